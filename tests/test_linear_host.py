"""Refusals of the linear layer's calls, without a GPU."""
import ctypes as C

import pytest
import torch

import fsdp_sharded_optimizer_step_amd as z
from fsdp_sharded_optimizer_step_amd import binding

EINVAL, ERANGE, EOVERLAP = binding.ZERO_EINVAL, binding.ZERO_ERANGE, binding.ZERO_EOVERLAP
O, I, T = 20, 30, 50
BIG = (1 << 24) + 1


@pytest.fixture(scope="module")
def L():
    return z.Layout([17, O * I, 24, O, 0], 0, 4, 1)


def at(n, off=0):
    """A host address standing in for a device pointer; never read."""
    return C.c_void_p(0x10000000 * n + off)


def good(L, name):
    h = L.handle
    return {
        "zero_linear": dict(L=h, tensor=1, tr=0, bias=3, params=at(1), x=at(2), xs=I, t=T, o=O, i=I, act=2, res=at(3),
                            rs=O, out=at(4), os=O, dtype=0, pre=at(5), ws=at(6), wb=1 << 22, stream=None),
        "zero_linear_input_grad": dict(L=h, tensor=1, tr=1, params=at(1), dy=at(2), ys=O, t=T, o=O, i=I, act=4,
                                       pre=at(3), add=at(4), adds=I, dx=at(5), xs=I, ws=at(6), wb=1 << 22, stream=None),
        "zero_bias_grad": dict(L=h, tensor=3, dy=at(1), ys=O, pre=at(2), act=1, t=T, scale=1.0, flags=0, dpre=at(3),
                               acc=at(4), out=at(5), ws=at(6), wb=1 << 20, stream=None),
    }[name]


def call(owner, name, **bad):
    args = dict(good(owner, name), **bad)
    return getattr(z.load(), name)(*args.values())


INF = float("inf")
BAD = [
    ("zero_linear", EINVAL, [
        dict(L=None), dict(tr=2), dict(o=21), dict(i=31), dict(o=-O, i=-I), dict(t=-1), dict(bias=-2), dict(bias=2),
        dict(act=5), dict(act=-1), dict(dtype=2), dict(params=None), dict(x=None), dict(out=None), dict(xs=I - 1),
        dict(os=O - 1), dict(rs=O - 1), dict(ws=None), dict(wb=100), dict(ws=at(6, 8)), dict(tensor=4, o=O, i=0)]),
    ("zero_linear", ERANGE, [dict(tensor=5), dict(tensor=-1), dict(bias=5), dict(t=(1 << 30) + 1), dict(xs=BIG),
                             dict(os=BIG), dict(rs=BIG), dict(o=(1 << 22) + 1)]),
    ("zero_linear", EOVERLAP, [dict(out=at(2)), dict(out=at(3)), dict(out=at(5)), dict(pre=at(2)), dict(ws=at(2)),
                               dict(out=at(1, 34)), dict(out=at(1, 2 * (17 + O * I + 24))), dict(pre=at(3, 10)),
                               dict(ws=at(4))]),
    ("zero_linear_input_grad", EINVAL, [
        dict(L=None), dict(tr=-1), dict(o=21), dict(t=-1), dict(act=9), dict(params=None), dict(dy=None),
        dict(dx=None), dict(ys=O - 1), dict(xs=I - 1), dict(adds=I - 1), dict(pre=None), dict(act=0), dict(ws=None),
        dict(wb=64), dict(ws=at(6, 4)), dict(tensor=4, o=0, i=I)]),
    ("zero_linear_input_grad", ERANGE, [dict(tensor=5), dict(t=(1 << 30) + 1), dict(ys=BIG), dict(xs=BIG),
                                        dict(adds=BIG)]),
    ("zero_linear_input_grad", EOVERLAP, [dict(dx=at(2)), dict(dx=at(3)), dict(dx=at(4)), dict(dx=at(1, 34)),
                                          dict(ws=at(5)), dict(ws=at(3))]),
    ("zero_bias_grad", EINVAL, [
        dict(L=None), dict(act=7), dict(act=0), dict(pre=None), dict(dy=None), dict(ys=O - 1), dict(t=-1),
        dict(scale=INF), dict(flags=8), dict(flags=4), dict(flags=2, out=None), dict(acc=None), dict(ws=None),
        dict(wb=8), dict(ws=at(6, 2))]),
    ("zero_bias_grad", ERANGE, [dict(tensor=5), dict(t=(1 << 30) + 1), dict(ys=BIG)]),
    ("zero_bias_grad", EOVERLAP, [dict(dpre=at(1)), dict(dpre=at(2)), dict(acc=at(1, -4 * (17 + O * I + 24))), dict(ws=at(1)),
                                  dict(flags=2, out=at(4, 2 * (17 + O * I + 24))), dict(ws=at(3))]),
]


@pytest.mark.parametrize("name,status,bads", BAD, ids=[f"{n}-{s}" for n, s, _ in BAD])
def test_the_library_refuses(L, name, status, bads):
    for bad in bads:
        assert call(L, name, **bad) == status, bad


def test_a_matrix_between_anothers_rows_is_refused(L):
    assert call(L, "zero_linear", xs=64, out=at(2, 2 * 32), os=64) == EOVERLAP
    assert call(L, "zero_linear_input_grad", ys=64, dx=at(2, 2 * 24), xs=64) == EOVERLAP
    assert call(L, "zero_bias_grad", ys=64, dpre=at(1, 2 * 24)) == EOVERLAP


def test_nothing_to_do(L):
    assert call(L, "zero_linear", t=0, x=None, out=None, ws=None) == 0
    assert call(L, "zero_linear", tensor=4, o=0, i=I, bias=-1, out=None) == 0
    assert call(L, "zero_linear_input_grad", t=0, dx=None) == 0
    assert call(L, "zero_linear_input_grad", tensor=4, o=O, i=0, dx=None) == 0
    assert call(L, "zero_bias_grad", t=0, dy=None, ws=None) == 0


def test_workspaces(L):
    """Copies of what is not aligned, and sums of what is split."""
    lib = z.load()
    f, g = lib.zero_linear_workspace, lib.zero_linear_input_grad_workspace
    al = z.Layout([16, 256 * 4096, 256 * 4100], 0, 4, 1)
    whole = f(al.handle, 1, 0, at(1), at(2), 4096, 1 << 20, 256, 4096)
    assert whole == 0
    assert f(al.handle, 1, 0, at(1), at(2, 2), 4096, 1 << 20, 256, 4096) == (1 << 20) * 4096 * 2
    assert f(al.handle, 1, 0, at(1, 2), at(2), 4096, 1 << 20, 256, 4096) == 256 * 4096 * 2
    assert f(al.handle, 2, 0, at(1), at(2), 4100, 1 << 20, 256, 4100) == (256 + (1 << 20)) * 4104 * 2
    assert g(al.handle, 1, 0, at(1), at(2), 256, 1 << 20, 256, 4096) == 0
    assert f(None, 1, 0, at(1), at(2), I, T, O, I) == EINVAL
    assert f(L.handle, 1, 0, at(1), at(2), I - 1, T, O, I) == EINVAL
    assert f(L.handle, 9, 0, at(1), at(2), I, T, O, I) == ERANGE
    assert f(L.handle, 1, 0, at(1), at(2), I, 0, O, I) == 0
    assert lib.zero_bias_grad_workspace(L.handle, 3, T) >= 4 * O
    assert lib.zero_bias_grad_workspace(L.handle, 3, 0) == 0 and lib.zero_bias_grad_workspace(L.handle, 7, 1) == ERANGE


def test_wrappers_refuse(L):
    b, f = torch.bfloat16, torch.float32
    new = lambda *s, dtype=b: torch.zeros(*s, dtype=dtype)  # noqa: E731
    params, x, out = new(L.padded), new(T, I), new(T, O)

    def fwd(params=params, x=x, out=out, tensor=1, **kw):
        z.zero_linear(L, tensor, params, x, out, **kw)
    for bad in (dict(x=new(T, I, dtype=f)), dict(x=new(T)), dict(out=new(T + 1, O)), dict(out=new(T, O, dtype=torch.float16)),
                dict(x=new(T, 2 * I)[:, ::2]), dict(params=new(L.padded - 1)), dict(params=new(L.padded, dtype=f)),
                dict(res=new(T, O + 1)), dict(pre=new(T, 2 * O)[:, :O]), dict(activation="tanh"),
                dict(res=new(T, O, dtype=f)), dict()):
        with pytest.raises(ValueError):
            fwd(**bad)
    for bad in (dict(tensor=9), dict(bias=9)):
        with pytest.raises(z.ZeroError):
            fwd(**bad)

    def grad(dy=out, dx=x, **kw):
        z.zero_linear_input_grad(L, 1, params, dy, dx, **kw)
    for bad in (dict(dy=new(T, O, dtype=f)), dict(dx=new(T - 1, I)), dict(dx=new(T, I, dtype=f)), dict(pre=x),
                dict(activation="gelu"), dict(activation="gelu", pre=new(T, I + 1)), dict(add=new(T, O)), dict()):
        with pytest.raises(ValueError):
            grad(**bad)

    def bias(dy=out, acc=new(L.padded, dtype=f), **kw):
        z.zero_bias_grad(L, 3, dy, acc, **kw)
    for bad in (dict(dy=x), dict(acc=None), dict(acc=new(L.padded)), dict(flags=2), dict(pre=out),
                dict(activation="silu"), dict(dpre=x), dict(dpre=new(T, O, dtype=f)), dict()):
        with pytest.raises(ValueError):
            bias(**bad)
