"""The step with 8-bit moments without a GPU: its refusals, and the references
that the GPU tests use."""
import ctypes as C

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_step_amd as z
import moments8_ref as ref
from fsdp_sharded_optimizer_step_amd import binding
from fsdp_sharded_optimizer_step_amd.binding import _AdamW

EINVAL, ERANGE, EOVERLAP = binding.ZERO_EINVAL, binding.ZERO_ERANGE, binding.ZERO_EOVERLAP
NAN = float("nan")


def at(n):
    """A host address standing in for a device pointer; never read."""
    return C.c_void_p(0x10000000 * n)


@pytest.fixture(scope="module")
def L():
    return z.Layout([17, 600, 24], 100, 4, 1)


def good(L, name):
    if name == "zero_shard_step_moments8":
        return dict(L=L.handle, hp=C.byref(z.AdamW()._c()), t=1, b0=0, b1=L.n_buckets,
                    g=(C.c_void_p * 4)(*[at(20 + q) for q in range(4)]), dtype=0, layout=0, master=at(1), mq=at(2),
                    me=at(3), vq=at(4), ve=at(5), out=at(6), mode=1, seed=1, stream=None)
    args = [("m", at(1)), ("v", at(2)), ("mq", at(3)), ("me", at(4)), ("vq", at(5)), ("ve", at(6))]
    if name == "zero_moments8_unpack":
        args = args[2:] + args[:2]
    return dict([("L", L.handle)] + args + [("stream", None)])


def call(owner, name, **bad):
    args = dict(good(owner, name), **bad)
    return getattr(z.load(), name)(*args.values())


def hp(**kw):
    return C.byref(z.AdamW(**kw)._c())


BAD = [
    ("zero_shard_step_moments8", EINVAL, [
        dict(L=None), dict(hp=None), dict(t=0), dict(hp=hp(lr=NAN)), dict(hp=hp(beta1=1.0)), dict(g=None),
        dict(g=(C.c_void_p * 4)(at(20), None, at(22), at(23))), dict(dtype=2), dict(layout=2), dict(master=None),
        dict(mq=None), dict(me=None), dict(vq=None), dict(ve=None), dict(out=None), dict(mode=3)]),
    ("zero_shard_step_moments8", ERANGE, [dict(b0=-1), dict(b1=8), dict(b0=3, b1=2)]),
    ("zero_shard_step_moments8", EOVERLAP, [
        dict(mq=at(1)), dict(vq=at(2)), dict(me=at(5)), dict(out=at(4)), dict(master=at(22)),
        dict(ve=C.c_void_p(at(21).value + 10))]),
    ("zero_moments8_pack", EINVAL, [dict(L=None), dict(m=None), dict(v=None), dict(mq=None), dict(me=None),
                                    dict(vq=None), dict(ve=None)]),
    ("zero_moments8_pack", EOVERLAP, [dict(mq=at(1)), dict(vq=at(3)), dict(me=at(2)), dict(ve=at(4))]),
    ("zero_moments8_unpack", EINVAL, [dict(L=None), dict(m=None), dict(v=None), dict(mq=None), dict(me=None),
                                      dict(vq=None), dict(ve=None)]),
    ("zero_moments8_unpack", EOVERLAP, [dict(m=at(2)), dict(v=at(3)), dict(m=at(4)), dict(v=at(6))]),
]


@pytest.mark.parametrize("name,status,bads", BAD, ids=[f"{n}-{s}" for n, s, _ in BAD])
def test_the_library_refuses(L, name, status, bads):
    for bad in bads:
        assert call(L, name, **bad) == status, bad


def test_nothing_to_do():
    L = z.Layout([17, 600, 24], 100, 4, 1)
    assert call(L, "zero_shard_step_moments8", b0=2, b1=2, master=None) == 0
    for empty in (z.Layout([], 0, 4, 1), z.Layout([0, 0], 0, 4, 1), z.Layout([0], 0, 2, 0, rows=[0])):
        assert empty.moment_blocks == 0
        assert call(empty, "zero_shard_step_moments8", b1=0, master=None, mq=None) == 0
        assert call(empty, "zero_moments8_pack", m=None) == 0
        assert call(empty, "zero_moments8_unpack", m=None) == 0


def test_blocks():
    assert z.load().zero_layout_moment_blocks(None) == -1
    assert z.Layout([1], 0, 8, 0).moment_blocks == 1
    assert z.Layout([8 * 128], 0, 8, 0).moment_blocks == 1
    assert z.Layout([8 * 128 + 1], 0, 8, 0).moment_blocks == 2
    assert z.Layout([1000], 300, 2, 0).moment_blocks == 3 * 2 + 1       # slices of 150, and 50
    assert z.Layout([4 * 200, 3], 0, 4, 0, rows=[4, 3]).moment_blocks == 2 + 1


def test_wrappers_refuse(L):
    new = lambda n, dtype=torch.uint8: torch.zeros(n, dtype=dtype)  # noqa: E731
    n, b = L.shard, L.moment_blocks
    f, mom = torch.float32, z.Moments8.zeros(L, "cpu")
    grads = [new(n, torch.bfloat16) for _ in range(4)]

    def step(grads=grads, master=new(n, f), moments=mom, out=new(n, torch.bfloat16)):
        z.zero_shard_step_moments8(L, z.AdamW(), 1, grads, z.GRAD_COMPACT, master, moments, out, z.OUT_SHARD, 0)
    for bad in (dict(grads=grads[:3]), dict(grads=grads[:3] + [new(n, f)]), dict(grads=[new(n)] * 4),
                dict(grads=grads[:3] + [new(n - 1, torch.bfloat16)]), dict(master=new(n)),
                dict(master=new(n - 1, f)), dict(master=new(2 * n, f)[::2]), dict(out=new(n, f)),
                dict(out=new(n - 1, torch.bfloat16)),
                dict(moments=z.Moments8(new(n - 1), new(b), new(n), new(b))),
                dict(moments=z.Moments8(new(n), new(b), new(n), new(b - 1))),
                dict(moments=z.Moments8(new(n), new(b, torch.int8), new(n), new(b))),
                dict()):                               # a host's tensors
        with pytest.raises(ValueError):
            step(**bad)
    for f_ in (lambda m, v, q: z.zero_moments8_pack(L, m, v, q), lambda m, v, q: z.zero_moments8_unpack(L, q, m, v)):
        for m, v, q in ((new(n - 1, f), new(n, f), mom), (new(n, f), new(n), mom), (new(n, f), new(n, f), mom)):
            with pytest.raises(ValueError):
                f_(m, v, q)


def test_reference_tables():
    assert ref.check_against_act8()
    x = (ref.V8[1:] * 2.0 ** 3).astype(np.float32)
    for lo in range(0, 254, 127):
        c, e = ref.encode("v", np.append(x[lo:lo + 127], x[-1]))
        assert np.array_equal(c[:-1], np.arange(1 + lo, 1 + lo + min(127, 254 - lo)))
    assert isinstance(z.AdamW()._c(), _AdamW)


def test_random_bits_are_even():
    """Mean and neighbours' products of 2^18 draws, within 5 standard deviations."""
    n = 1 << 18
    h = ref.random_bits(1, 1, np.arange(n))
    for x in (h & np.uint64(0xFFFF), h >> np.uint64(16)):
        u = (x.astype(np.float64) + 0.5) / 65536 - 0.5
        assert abs(u.mean()) * (12 * n) ** 0.5 < 5
        for k in (1, 2, 4, 128, 256):
            assert abs((u[k:] * u[:-k]).mean()) * 12 * n ** 0.5 < 5
