"""Refusals of the micro-batch operators, without a GPU: the library's own
checks through its C entry points (nothing is launched: every call here ends
before that), and the Python wrappers' checks of shapes, types and devices."""
import ctypes as C

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_step_amd as z
from fsdp_sharded_optimizer_step_amd import binding
from micrograd_ref import E4M3, act8, act8_values

EINVAL, ERANGE, EOVERLAP = binding.ZERO_EINVAL, binding.ZERO_ERANGE, binding.ZERO_EOVERLAP
NUMEL = [17, 600, 24]                      # tensor 1: 20 x 30 table / weight, tensor 2: a norm
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    return z.Layout(NUMEL, 0, 4, 1)


def at(n):
    """A host address standing in for a device pointer; never read."""
    return C.c_void_p(0x10000000 * n)


def call(name, good, **bad):
    """Status of the entry point with the good arguments but for `bad`."""
    args = dict(good, **bad)
    assert set(args) == set(good)
    return getattr(z.load(), name)(*args.values())


def good_calls(L):
    h = L.handle
    return {
        "zero_act8_pack": dict(x=at(1), dtype=0, rows=5, cols=200, stride=200, codes=at(2),
                               scales=at(3), stream=None),
        "zero_act8_unpack": dict(codes=at(2), scales=at(3), rows=5, cols=200, x=at(1), dtype=1,
                                 stride=200, stream=None),
        "zero_embedding_lookup": dict(L=h, tensor=1, cols=30, params=at(1), ids=at(2), id_bytes=8,
                                      n=9, scale=1.0, out=at(3), stride=30, dtype=0, stream=None),
        "zero_embedding_grad": dict(L=h, tensor=1, cols=30, ids=at(2), id_bytes=8, n=900, dy=at(3),
                                    stride=30, dtype=0, scale=1.0, flags=0, acc=at(4), out=at(5),
                                    ws=at(6), ws_bytes=1 << 20, stream=None),
        "zero_rms_norm": dict(L=h, tensor=2, params=at(1), x=at(2), stride=24, res=at(3),
                              res_stride=24, rows=5, eps=1e-5, h=at(4), rstd=at(5), codes=at(6),
                              scales=at(7), y=at(8), stream=None),
        "zero_rms_norm_grad": dict(L=h, tensor=2, params=at(1), dy=at(2), stride=24, dh=at(3),
                                   dh_stride=24, h=at(4), rstd=at(5), rows=5, scale=1.0, flags=0,
                                   dx=at(6), acc=at(7), out=at(8), ws=at(9), ws_bytes=1 << 20,
                                   stream=None),
        "zero_linear_grad": dict(L=h, tensor=1, tr=0, dy=at(1), stride=20, codes=at(2),
                                 scales=at(3), tokens=4000, o=20, i=30, scale=1.0, flags=0,
                                 acc=at(4), out=at(5), ws=at(6), ws_bytes=1 << 20, stream=None),
    }


INF = float("inf")
BAD = [
    ("zero_act8_pack", EINVAL, [dict(x=None), dict(codes=None), dict(scales=None), dict(dtype=2),
                                dict(rows=-1), dict(cols=-1), dict(stride=199)]),
    ("zero_act8_pack", ERANGE, [dict(rows=(1 << 30) + 1), dict(stride=(1 << 24) + 1),
                                dict(cols=(1 << 24) + 1, stride=BIG)]),
    ("zero_act8_pack", EOVERLAP, [dict(codes=at(1)), dict(scales=at(2))]),
    ("zero_act8_unpack", EINVAL, [dict(x=None), dict(codes=None), dict(dtype=-1), dict(stride=10)]),
    ("zero_act8_unpack", EOVERLAP, [dict(x=at(2)), dict(x=at(3))]),
    ("zero_embedding_lookup", EINVAL, [
        dict(L=None), dict(cols=0), dict(cols=31), dict(n=-1), dict(id_bytes=2), dict(dtype=5),
        dict(scale=INF), dict(ids=None), dict(out=None), dict(params=None), dict(stride=29)]),
    ("zero_embedding_lookup", ERANGE, [dict(tensor=3), dict(tensor=-1), dict(n=(1 << 30) + 1),
                                       dict(stride=BIG)]),
    ("zero_embedding_lookup", EOVERLAP, [dict(out=at(2)), dict(out=C.c_void_p(at(1).value + 40))]),
    ("zero_embedding_grad", EINVAL, [
        dict(L=None), dict(cols=7), dict(n=-1), dict(id_bytes=1), dict(dtype=2), dict(scale=INF),
        dict(ids=None), dict(dy=None), dict(stride=29), dict(acc=None), dict(flags=8),
        dict(flags=4), dict(flags=2, out=None), dict(ws=None), dict(ws_bytes=64),
        dict(ws=C.c_void_p(at(6).value + 8))]),
    ("zero_embedding_grad", ERANGE, [dict(tensor=7), dict(n=(1 << 30) + 1)]),
    ("zero_embedding_grad", EOVERLAP, [dict(dy=C.c_void_p(at(4).value + 68)), dict(ws=at(3)),
                                       dict(flags=2, out=at(4))]),
    ("zero_rms_norm", EINVAL, [
        dict(L=None), dict(params=None), dict(x=None), dict(rows=-1), dict(eps=-1.0),
        dict(eps=INF), dict(eps=float("nan")), dict(h=None), dict(rstd=None), dict(codes=None),
        dict(scales=None), dict(stride=23), dict(res_stride=23)]),
    ("zero_rms_norm", ERANGE, [dict(tensor=3), dict(rows=(1 << 30) + 1), dict(stride=BIG),
                               dict(res_stride=BIG)]),
    ("zero_rms_norm", EOVERLAP, [dict(h=at(3)), dict(y=at(4)), dict(codes=at(2)), dict(rstd=at(7)),
                                 dict(scales=C.c_void_p(at(1).value + 2 * 617))]),
    ("zero_rms_norm_grad", EINVAL, [
        dict(L=None), dict(params=None), dict(dy=None), dict(h=None), dict(rstd=None),
        dict(dx=None), dict(acc=None), dict(rows=-1), dict(stride=23), dict(dh_stride=23),
        dict(scale=INF), dict(flags=16), dict(flags=4), dict(flags=3, out=None), dict(ws=None),
        dict(ws_bytes=10), dict(ws=C.c_void_p(at(9).value + 4))]),
    ("zero_rms_norm_grad", ERANGE, [dict(tensor=3), dict(rows=(1 << 30) + 1), dict(stride=BIG)]),
    ("zero_rms_norm_grad", EOVERLAP, [dict(dx=at(2)), dict(dx=at(3)), dict(dx=at(4)),
                                      dict(ws=at(2)),
                                      dict(flags=2, out=C.c_void_p(at(7).value + 2 * 617))]),
    ("zero_linear_grad", EINVAL, [
        dict(L=None), dict(tr=2), dict(dy=None), dict(codes=None), dict(scales=None),
        dict(stride=19), dict(o=21), dict(i=31), dict(tokens=-1), dict(o=-20, i=-30),
        dict(scale=INF), dict(flags=8), dict(flags=4), dict(flags=2, out=None), dict(acc=None),
        dict(ws=None), dict(ws_bytes=16), dict(ws=C.c_void_p(at(6).value + 4))]),
    ("zero_linear_grad", ERANGE, [dict(tensor=3), dict(tokens=(1 << 30) + 1), dict(stride=BIG),
                                  dict(o=(1 << 24) + 1)]),
    ("zero_linear_grad", EOVERLAP, [dict(acc=at(1)), dict(ws=at(2)), dict(flags=2, out=at(4))]),
]


@pytest.mark.parametrize("name,status,bads", BAD, ids=[f"{n}-{s}" for n, s, _ in BAD])
def test_the_library_refuses(L, name, status, bads):
    good = good_calls(L)[name]
    for bad in bads:
        assert call(name, good, **bad) == status, bad


@pytest.mark.parametrize("name", ["zero_act8_pack", "zero_act8_unpack", "zero_embedding_lookup",
                                  "zero_embedding_grad", "zero_rms_norm", "zero_rms_norm_grad",
                                  "zero_linear_grad"])
def test_nothing_to_do_needs_no_buffers(L, name):
    """No rows and nothing to overwrite: accepted, nothing is touched."""
    good = good_calls(L)[name]
    empty = {k: (None if isinstance(v, C.c_void_p) and k not in ("L", "acc") else v)
             for k, v in good.items()}
    for k in ("rows", "n", "tokens"):
        if k in empty:
            empty[k] = 0
    assert call(name, empty) == binding.ZERO_OK


def test_workspace_queries(L):
    lib, h = z.load(), L.handle
    assert lib.zero_embedding_grad_workspace(h, 1, 30, 512, 0) == 0     # few tokens, added
    assert lib.zero_embedding_grad_workspace(h, 1, 30, 512, 2) >= 512 * 16
    assert lib.zero_embedding_grad_workspace(h, 1, 30, 513, 0) >= 513 * 16
    assert lib.zero_embedding_grad_workspace(h, 1, 31, 9, 0) == EINVAL
    assert lib.zero_embedding_grad_workspace(h, 9, 30, 9, 0) == ERANGE
    assert lib.zero_rms_norm_grad_workspace(h, 2, 5) >= 24 * 4
    assert lib.zero_rms_norm_grad_workspace(None, 2, 5) == EINVAL
    assert lib.zero_linear_grad_workspace(h, 1, 0, 20, 30, 4000) >= 600 * 4
    assert lib.zero_linear_grad_workspace(h, 1, 0, 20, 31, 4000) == EINVAL
    assert lib.zero_linear_grad_workspace(h, 1, 3, 20, 30, 4000) == EINVAL


def test_norm_width_limit():
    wide = z.Layout([32769], 0, 1, 0)
    assert z.load().zero_rms_norm_grad_workspace(wide.handle, 0, 1) == ERANGE


# ------------------------------------------------------------------ wrappers
def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def wrapper_calls(L):
    P = L.padded
    f, u8 = torch.float32, torch.uint8
    a = dict(params=t(P), acc=t(P, dtype=f), out=t(P))
    return {
        "pack": (z.zero_act8_pack, [t(5, 200), t(5, 200, dtype=u8), t(5, 2, dtype=u8)]),
        "unpack": (z.zero_act8_unpack, [t(5, 200, dtype=u8), t(5, 2, dtype=u8), t(5, 200, dtype=f)]),
        "lookup": (z.zero_embedding_lookup, [L, 1, a["params"], t(9, dtype=torch.int64), t(9, 30)]),
        "emb_grad": (z.zero_embedding_grad, [L, 1, t(9, dtype=torch.int32), t(9, 30), a["acc"], 1.0,
                                             2, a["out"]]),
        "norm": (z.zero_rms_norm, [L, 2, a["params"], t(5, 24), t(5, 24), 1e-5, t(5, 24),
                                   t(5, dtype=f), t(5, 24, dtype=u8), t(5, 1, dtype=u8), t(5, 24)]),
        "norm_grad": (z.zero_rms_norm_grad, [L, 2, a["params"], t(5, 24), t(5, 24), t(5, 24),
                                             t(5, dtype=f), t(5, 24), a["acc"], 1.0, 2, a["out"]]),
        "linear": (z.zero_linear_grad, [L, 1, t(50, 20), t(50, 30, dtype=u8), t(50, 1, dtype=u8),
                                        a["acc"], 1.0, 2, a["out"]]),
    }


@pytest.mark.parametrize("name", ["pack", "unpack", "lookup", "emb_grad", "norm", "norm_grad",
                                  "linear"])
def test_wrappers_check_types_shapes_and_devices(L, name):
    fn, args = wrapper_calls(L)[name]
    with pytest.raises(ValueError, match="CUDA tensors"):
        fn(*args)
    for k, v in enumerate(args):
        if not torch.is_tensor(v):
            continue
        wrong_type = v.to(torch.float64)
        wrong_shape = v[:-1] if v.numel() > 1 else v.repeat(2)
        for w in (wrong_type, wrong_shape):
            with pytest.raises(ValueError) as err:
                fn(*args[:k], w, *args[k + 1:])
            assert "needs CUDA tensors" not in str(err.value), (k, str(err.value))


def test_wrappers_refuse_columns_that_are_not_adjacent_and_missing_outputs(L):
    for name in ("pack", "lookup", "emb_grad", "norm", "linear"):
        fn, args = wrapper_calls(L)[name]
        k = {"pack": 0, "lookup": 4, "emb_grad": 3, "norm": 3, "linear": 2}[name]
        m = args[k]
        with pytest.raises(ValueError, match="adjacent"):
            fn(*args[:k], m.t().contiguous().t(), *args[k + 1:])
        with pytest.raises(ValueError, match="rows overlap"):
            fn(*args[:k], m[:1].expand(m.shape), *args[k + 1:])
    fn, args = wrapper_calls(L)["emb_grad"]
    with pytest.raises(ValueError, match="bf16_out is needed"):
        fn(*args[:7])
    with pytest.raises(ValueError, match="acc is needed"):
        fn(*args[:4], None, 1.0, 0)
    with pytest.raises(z.ZeroError):
        fn(L, 3, *args[2:])


# ------------------------------------------------------------------ the references themselves
def test_reference_codes_agree_with_the_type_of_torch():
    """The reference's rounding against torch's e4m3 conversion on the CPU."""
    assert np.array_equal(E4M3, torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn)
                          .double().numpy())
    x = torch.randn(40, 300, generator=torch.Generator().manual_seed(0)) * 5
    codes, scales = act8(x.double().numpy())
    s = torch.exp2(torch.from_numpy(scales).double() - 127).repeat_interleave(128, 1)[:, :300]
    exp = (x.double() / s).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(codes, exp)
    v = act8_values(codes, scales)
    assert np.abs(v - x.double().numpy()).max() <= 2.0 ** -4 * np.abs(x.numpy()).max()
    bf = torch.from_numpy(v).to(torch.bfloat16).double().numpy()
    assert np.array_equal(bf, v)


# ------------------------------------------------------------------ very large weights
@pytest.mark.parametrize("o,i", [(300, 1 << 24), (1 << 24, 130), (1 << 17, 1 << 18), (129, 1 << 24)])
def test_weights_of_up_to_2_35_elements_are_accepted(o, i):
    """Checked by the one refusal that comes after all others: an overlap."""
    big = z.Layout([o * i], 0, 1, 0)
    lib = z.load()
    for tr in (0, 1):
        for tokens in (1, 1000):
            size = lib.zero_linear_grad_workspace(big.handle, 0, tr, o, i, tokens)
            assert size >= 0
            assert lib.zero_linear_grad(big.handle, 0, tr, at(1), o, at(1 << 20), at(1 << 21), tokens, o, i,
                                        1.0, 0, at(1), None, at(1 << 22), size, None) == EOVERLAP


def test_larger_weights_are_refused_by_the_call_and_its_workspace_alike():
    o = i = 1 << 24
    big = z.Layout([o * i], 0, 1, 0)
    lib = z.load()
    assert lib.zero_linear_grad_workspace(big.handle, 0, 0, o, i, 5) == ERANGE
    assert lib.zero_linear_grad(big.handle, 0, 0, at(1), o, at(2), at(3), 5, o, i, 1.0, 0, at(4), None,
                                None, 0, None) == ERANGE


def test_wrappers_take_empty_batches_whatever_their_strides(L):
    """An empty array's strides say nothing (numpy's are zero in torch)."""
    for name in ("pack", "lookup", "emb_grad", "norm", "norm_grad", "linear"):
        fn, args = wrapper_calls(L)[name]
        rows = {"pack": 5, "lookup": 9, "emb_grad": 9, "norm": 5, "norm_grad": 5, "linear": 50}[name]
        none = []
        for v in args:
            if torch.is_tensor(v) and v.shape[0] == rows:
                v = v[:0].as_strided((0, *v.shape[1:]), (0,) * v.dim())
            none.append(v)
        with pytest.raises(ValueError, match="needs CUDA tensors"):
            fn(*none)
