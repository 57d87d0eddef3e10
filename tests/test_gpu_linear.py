"""The linear layer, the gradient of its input and of its bias on the GPU,
against 64-bit references.

Tolerances.  U = 2^-24, BF = 2^-8 (half a step of binary32 and of bf16).  A sum
of K exact products in any order is off by K U times the sum of their
magnitudes at most; bias, addend and the activation's argument add a rounding
each.  An activation or its derivative is computed from a binary32 argument p
within 64 U (1 + |p|): the functions' own 2 to 8 units of the last place, and
an argument of exp or erfc that is off by 8 U of itself, which moves the value
by 8 U |z f'(z)|, below 8 U |p| for all of them.  Its argument's error passes
on with the largest slope, 1.13.  Small whole numbers have exact sums.
"""
import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_step_amd as z
import oracle
from linear_cases import LARGE_TILES
from micrograd_ref import BF, FLAG_SETS, U, Flat, f64
from micrograd_ref import layout as odd_layout
from test_gpu_micrograd import randn, strided

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(autouse=True)
def _free_gpu_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def ints(seed, *shape, top=4):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-top, top + 1, shape, generator=g, device=DEV).to(BF16)


def act64(x, act):
    x = x.double()
    if act == "relu":
        return torch.where(x > 0, x, 0.0)
    if act == "gelu":
        return x * torch.special.ndtr(x)
    if act == "gelu_tanh":
        return x * torch.sigmoid(2 * (2 / np.pi) ** 0.5 * (x + 0.044715 * x ** 3))
    return x * torch.sigmoid(x) if act == "silu" else x


def slope64(x, act):
    if act == "none":
        return torch.ones_like(x, dtype=torch.float64)
    y = x.double().requires_grad_()
    (g,) = torch.autograd.grad(act64(y, act).sum(), y)
    return g


class Weights:
    """A layout [lead, out * in, 3, out], its flat parameters, and W and b in 64 bits."""

    def __init__(self, o, i, tr, lead=16, cap=0, n_d=4, fill=None):
        self.sizes = [lead, o * i, 3, o]
        self.L = z.Layout(self.sizes, cap, n_d, 0)
        pl = oracle.plan(self.sizes, cap, n_d)
        self.params = (fill or (lambda n: randn(n % 97, n)))(self.L.padded)

        def place(first, n):
            x = first + np.arange(n)
            b = np.searchsorted(pl.stream_off, x, side="right") - 1
            return torch.from_numpy(np.asarray(pl.padded_off)[b] + x - np.asarray(pl.stream_off)[b]).to(DEV)
        w = self.params[place(lead, o * i)].double()
        self.w = (w.view(i, o).t() if tr else w.view(o, i)).contiguous()
        self.b = self.params[place(lead + o * i + 3, o)].double()


SHAPES = [(1, 1, 1), (1, 8, 8), (3, 5, 7), (2, 16, 40), (31, 24, 64), (127, 129, 65), (128, 128, 64), (129, 264, 72),
          (33, 72, 129), (256, 256, 128), (300, 520, 200), (5, 1000, 1000), (16, 2048, 512), (17, 512, 2056),
          (70, 333, 4097), (513, 512, 1024), (1000, 2304, 768), (4100, 1032, 136), (3000, 4096, 320)]


@pytest.mark.parametrize("tr", [False, True])
@pytest.mark.parametrize("t,o,i", SHAPES)
def test_whole_numbers(t, o, i, tr):
    """Every product and every place: sums of whole numbers are exact."""
    w = Weights(o, i, tr, fill=lambda n: ints(n, n))
    x, dy = ints(1, t, i), ints(2, t, o)
    res, pre = ints(3, t, o, top=100), torch.zeros(t, o, dtype=BF16, device=DEV)
    out = torch.zeros(t, o, dtype=F32, device=DEV)
    z.zero_linear(w.L, 1, w.params, x, out, bias=3, res=res, pre=pre, transposed=tr)
    p = x.double() @ w.w.t() + w.b
    assert torch.equal(out.double(), p + res.double())
    assert torch.equal(pre, p.float().bfloat16())
    dx, add = torch.zeros(t, i, dtype=BF16, device=DEV), ints(4, t, i, top=100)
    z.zero_linear_input_grad(w.L, 1, w.params, dy, dx, add=add, transposed=tr)
    assert torch.equal(dx, (dy.double() @ w.w + add.double()).float().bfloat16())


@pytest.mark.parametrize("tr", [False, True])
@pytest.mark.parametrize("t,o,i", [(5, 40, 24), (130, 136, 264), (61, 77, 129), (700, 260, 320)])
@pytest.mark.parametrize("how", ["odd place", "padding inside", "odd rows", "odd start", "columns of more"])
def test_addresses(how, t, o, i, tr):
    """Operands that begin anywhere, with rows of any distance."""
    n_d, cap = 4, 0
    if how == "padding inside":
        cap = o * i // 3 // n_d * n_d + 1
    w = Weights(o, i, tr, lead=17 if how == "odd place" else 16, cap=cap, n_d=n_d, fill=lambda n: ints(n, n))
    extra, off = {"odd rows": (3, 0), "odd start": (8, 5), "columns of more": (64, 8)}.get(how, (0, 0))
    x, dy = strided(ints(1, t, i), extra, off), strided(ints(2, t, o), extra, off)
    res, add = strided(ints(3, t, o), extra, off), strided(ints(4, t, i), extra, off)
    out = strided(torch.zeros(t, o, dtype=F32, device=DEV), extra, off)
    z.zero_linear(w.L, 1, w.params, x, out, bias=3, res=res, transposed=tr)
    assert torch.equal(out.double(), x.double() @ w.w.t() + w.b + res.double())
    dx = strided(torch.zeros(t, i, dtype=BF16, device=DEV), extra, off)
    z.zero_linear_input_grad(w.L, 1, w.params, dy, dx, add=add, transposed=tr)
    assert torch.equal(dx, (dy.double() @ w.w + add.double()).float().bfloat16())
    for v, cols in ((out, o), (dx, i)):
        if extra:
            assert (v.as_strided((t, cols + extra), (cols + extra, 1))[:-1, cols:] == 7).all()


@pytest.mark.parametrize("tr", [False, True])
@pytest.mark.parametrize("t", list(range(1, 10)) + [15, 16, 17])
def test_few_tokens(t, tr):
    """One pass over the weight up to 16 tokens (4 where the sums run down its
    columns), at odd places, across padding, for lengths around a wave's."""
    for o, i, lead, cap in ((1, 700, 17, 0), (65, 63, 17, 0), (200, 1024 + 9, 16, 0), (513, 64, 5, 4001), (16, 2000, 16, 0)):
        w = Weights(o, i, tr, lead=lead, cap=cap, fill=lambda n: ints(n, n))
        x, dy = strided(ints(1, t, i), 5, 3), strided(ints(2, t, o), 1, 0)
        res, pre = ints(3, t, o, top=50), torch.zeros(t, o, dtype=BF16, device=DEV)
        out = strided(torch.zeros(t, o, dtype=F32, device=DEV), 2, 1)
        z.zero_linear(w.L, 1, w.params, x, out, bias=3, res=res, pre=pre, transposed=tr, activation="relu")
        p = x.double() @ w.w.t() + w.b
        assert torch.equal(out.double(), p.clamp(min=0) + res.double())
        assert torch.equal(pre, p.float().bfloat16())
        dx, add = strided(torch.zeros(t, i, dtype=BF16, device=DEV), 3, 1), ints(4, t, i, top=50)
        z.zero_linear_input_grad(w.L, 1, w.params, dy, dx, activation="relu", pre=x.contiguous(), add=add, transposed=tr)
        assert torch.equal(dx, torch.where(x > 0, dy.double() @ w.w + add.double(), 0.0).float().bfloat16())
        assert (out.as_strided((t, o + 2), (o + 2, 1))[:-1, o:] == 7).all()


@pytest.mark.parametrize("lead", [16, 17])
@pytest.mark.parametrize("tr", [False, True])
@pytest.mark.parametrize("o,i", [(64, 9000), (2048, 8192), (4096, 8200), (500, 16384), (16400, 512), (20000, 2048),
                                 (8200, 1024), (8192, 1024), (4096, 2056)])
def test_few_tokens_on_both_sides_of_the_choice(o, i, tr, lead):
    """Sizes next to where other kernels take few tokens' products, with and
    without a copy of the weight, forward and as the gradient of the other order."""
    w = Weights(o, i, tr, lead=lead, fill=lambda n: ints(n, n))
    for t in (1, 2, 3, 5, 8, 9, 16):
        x, dy = ints(t, t, i), ints(t + 1, t, o)
        out = torch.zeros(t, o, dtype=F32, device=DEV)
        z.zero_linear(w.L, 1, w.params, x, out, bias=3, transposed=tr)
        assert torch.equal(out.double(), x.double() @ w.w.t() + w.b)
        dx = torch.zeros(t, i, dtype=BF16, device=DEV)
        z.zero_linear_input_grad(w.L, 1, w.params, dy, dx, transposed=tr)
        assert torch.equal(dx, (dy.double() @ w.w).float().bfloat16())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("t,o,i,tr", [(1, 512, 300, False), (40, 260, 512, True), (300, 384, 256, False),
                                      (2100, 1024, 192, True)])
def test_epilogues(act, t, o, i, tr):
    w = Weights(o, i, tr, fill=lambda n: randn(n % 89, n, scale=i ** -0.5))
    x, res = randn(1, t, i, scale=3.0), randn(2, t, o)
    out, pre = torch.empty(t, o, dtype=BF16, device=DEV), torch.empty(t, o, dtype=BF16, device=DEV)
    z.zero_linear(w.L, 1, w.params, x, out, bias=3, activation=act, res=res, pre=pre, transposed=tr)
    p = x.double() @ w.w.t() + w.b
    mag = x.double().abs() @ w.w.abs().t() + w.b.abs()
    ep = (i + 2) * U * mag
    assert ((pre.double() - p).abs() <= ep + BF * (p.abs() + ep)).all()
    y = act64(p, act) + res.double()
    ey = 1.13 * ep + (0 if act == "none" else 64 * U * (1 + p.abs())) + 2 * U * (y.abs() + res.double().abs())
    assert ((out.double() - y).abs() <= ey + BF * (y.abs() + ey)).all()
    # the gradient of what an activation made the input from
    dy, add = randn(3, t, o, scale=0.1), randn(4, t, i, scale=0.1)
    before = randn(5, t, i, scale=3.0)
    dx = torch.empty(t, i, dtype=BF16, device=DEV)
    z.zero_linear_input_grad(w.L, 1, w.params, dy, dx, activation=act, pre=before if act != "none" else None, add=add,
                             transposed=tr)
    g = dy.double() @ w.w + add.double()
    eg = (o + 2) * U * (dy.double().abs() @ w.w.abs() + add.double().abs())
    s = slope64(before, act)
    es = 0 if act == "none" else 64 * U * (1 + before.double().abs())
    e = eg * (s.abs() + es) + g.abs() * es + 2 * U * (g * s).abs()
    assert ((dx.double() - g * s).abs() <= e + BF * ((g * s).abs() + e) + 2.0 ** -134).all()


@pytest.mark.parametrize("act", ACTS)
def test_activations_at_every_bf16_value(act):
    """W = 1: the activation and its derivative of every finite bf16 number."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.uint16).view(BF16).to(DEV)
    x = x[torch.isfinite(x)].view(-1, 1).contiguous()
    w = Weights(1, 1, False, fill=lambda n: torch.ones(n, dtype=BF16, device=DEV))
    out = torch.empty(x.shape, dtype=F32, device=DEV)
    z.zero_linear(w.L, 1, w.params, x, out, activation=act)
    y = act64(x, act)
    assert ((out.double() - y).abs() <= 64 * U * torch.clamp(y.abs(), min=2.0 ** -126) + 64 * U * x.double().abs()).all()
    if act == "none":
        return
    dx = torch.empty_like(x)
    z.zero_linear_input_grad(w.L, 1, w.params, torch.ones_like(x), dx, activation=act, pre=x)
    s = slope64(x.cpu(), act).to(DEV) if act != "gelu_tanh" else None
    if s is None:                               # its 64-bit form overflows for the largest numbers
        s = torch.where(x.abs() > 30, (x > 0).double(), slope64(x.clamp(-30, 30), act))
    assert ((dx.double() - s).abs() <= 64 * U * (1 + torch.clamp(x.double().abs(), max=40)) + BF * s.abs()).all()


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_activations_keep_their_digits_below_zero(act):
    """Every finite bf16 number below zero, relative to the value itself.

    e^a is off by the error of a, 2 U |a| for its product with log2(e), and 2 U.
    gelu: a = q - z^2 by 4 U z^2 (z is off by 2 U of itself), a rounding, the fit's
    1.5 U and q's 25 U (8 steps of magnitude 1.5, and t, which is off by 6 U of
    itself, with Q's slope of 2): 3.5 U x^2 + 44 U with the factors' roundings.
    gelu_tanh: a is off by 7 U of itself, silu: not at all; 1 / (1 + e^-a) adds 3
    roundings and the product one.  Factors below 2^-126 may be 0.
    The derivative of gelu adds x times the density, off by 1.5 U x^2 + 10 U of
    itself; those of the others a product of the same p with 1 - p, off by another
    U, and three roundings (of the polynomial in gelu_tanh another four)."""
    x = torch.arange(32769, 65536, dtype=torch.int32).to(torch.uint16).view(BF16).to(DEV)
    x = x[torch.isfinite(x)].view(-1, 1).contiguous()
    w = Weights(1, 1, False, fill=lambda n: torch.ones(n, dtype=BF16, device=DEV))
    out, dx = torch.empty(x.shape, dtype=F32, device=DEV), torch.empty_like(x)
    z.zero_linear(w.L, 1, w.params, x, out, activation=act)
    z.zero_linear_input_grad(w.L, 1, w.params, torch.ones_like(x), dx, activation=act, pre=x)
    v = x.double().clamp(min=-1000.0)          # all further ones are 0 in 64 bits, too
    a = {"gelu": v * v, "silu": v, "gelu_tanh": 2 * (2 / np.pi) ** 0.5 * (v + 0.044715 * v ** 3)}[act].abs()
    if act == "gelu":                           # ndtr is made of 1 + erf, which has no digits there
        low, dense = torch.special.erfc(-v * 0.5 ** 0.5) / 2, v * torch.exp(-v * v / 2) / (2 * np.pi) ** 0.5
        y, s, parts = v * low, low + dense, low + dense.abs()
        rel = (44 + 4 * a) * U
        rel_s = rel + 2 * U
    else:
        y, s = act64(v, act), slope64(v, act)
        rel = (12 + (10 if act == "gelu_tanh" else 3) * a) * U
        slope = 2 * (2 / np.pi) ** 0.5 * (1 + 0.134145 * v * v) if act == "gelu_tanh" else 1.0
        parts, rel_s = torch.sigmoid(-a) * (1 + v.abs() * slope), 2 * rel
    least = 2.0 ** -126 * x.double().abs() + 2.0 ** -149    # the second: the result's own step
    assert ((out.double() - y).abs() <= rel * y.abs() + least).all()
    e = rel_s * parts + 2.0 ** -126 * (1 + v.abs()) ** 3
    assert ((dx.double() - s).abs() <= e + BF * (s.abs() + e) + 2.0 ** -134).all()


def test_values_outside_the_matrices_count_for_nothing():
    """Infinities and NaN behind a row's last column, behind the last row, and in
    the parameters around the weight."""
    for o, i, lead in ((72, 40, 16), (70, 33, 17)):
        for tr in (False, True):
            w = Weights(o, i, tr, lead=lead, fill=lambda n: ints(n, n))
            around = w.params.clone()
            around[:lead], around[lead + o * i:lead + o * i + 3] = float("nan"), float("inf")
            x = torch.full((50, i + 24), float("nan"), dtype=BF16, device=DEV)
            x[:40, :i] = ints(1, 40, i)
            out = torch.empty(40, o, dtype=F32, device=DEV)
            z.zero_linear(w.L, 1, around, x[:40, :i], out, transposed=tr)
            assert torch.equal(out.double(), x[:40, :i].double() @ w.w.t())
            dy = torch.full((50, o + 24), float("inf"), dtype=BF16, device=DEV)
            dy[:40, :o] = ints(2, 40, o)
            dx = torch.empty(40, i, dtype=BF16, device=DEV)
            z.zero_linear_input_grad(w.L, 1, around, dy[:40, :o], dx, transposed=tr)
            assert torch.equal(dx, (dy[:40, :o].double() @ w.w).float().bfloat16())


def test_a_token_of_infinities_leaves_the_others_alone():
    w = Weights(200, 136, False, fill=lambda n: ints(n, n))
    x = ints(1, 150, 136)
    clean, out = (torch.empty(150, 200, dtype=F32, device=DEV) for _ in range(2))
    z.zero_linear(w.L, 1, w.params, x, clean)
    bad = x.clone()
    bad[7, 3], bad[140] = float("inf"), float("nan")
    z.zero_linear(w.L, 1, w.params, bad, out)
    ok = torch.ones(150, dtype=torch.bool, device=DEV)
    ok[7] = ok[140] = False
    assert torch.equal(clean[ok], out[ok]) and not torch.isfinite(out[140]).any()


def test_input_gradient_against_differences():
    """A loss's slope along a direction, by central differences of the 64-bit
    forward pass, is the gradient's product with it."""
    t, o, i = 20, 48, 56
    w = Weights(o, i, False, fill=lambda n: randn(n % 89, n, scale=0.2))
    pre, dy = randn(1, t, i), randn(2, t, o)
    v = torch.randn(t, i, dtype=torch.float64, device=DEV, generator=torch.Generator(DEV).manual_seed(0))
    dx = torch.empty(t, i, dtype=BF16, device=DEV)
    z.zero_linear_input_grad(w.L, 1, w.params, dy, dx, activation="gelu", pre=pre)
    h = 1e-5
    loss = lambda s: (dy.double() * (act64(pre.double() + s * v, "gelu") @ w.w.t())).sum()  # noqa: E731
    slope = (loss(h) - loss(-h)) / (2 * h)
    mag = ((dy.double().abs() @ w.w.abs()) * v.abs() * 1.13).sum()
    # rounding of dx; the difference's third derivative (below 4 v^3 h^2) and its cancellation
    bound = (BF * (dx.double() * v).abs()).sum() + (o + 70) * U * mag + 4 * h * h * mag * v.abs().max() ** 2 + 1e-10 * mag
    assert abs(float((dx.double() * v).sum() - slope)) <= float(bound)


# ------------------------------------------------------------------ bias gradient
@pytest.mark.parametrize("rows,cols,extra,off", [(1, 1, 0, 0), (3, 7, 1, 1), (17, 64, 0, 0), (200, 129, 3, 0),
                                                 (64, 520, 0, 0), (1000, 2304, 8, 3), (5000, 96, 0, 0), (333, 4099, 0, 0),
                                                 (20000, 8, 0, 0)])
@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_bias_gradient(rows, cols, extra, off, act):
    L, pl = odd_layout(cols, False)
    dy = strided(randn(rows, rows, cols), extra, off)
    pre = randn(cols, rows, cols, scale=3.0) if act != "none" else None
    flat, dpre = Flat(L, pl, cols, DEV, seed=rows), torch.empty(rows, cols, dtype=BF16, device=DEV)
    z.zero_bias_grad(L, 1, dy, flat.acc, -0.5, activation=act, pre=pre, dpre=dpre)
    s = slope64(pre, act) if act != "none" else 1.0
    es = 64 * U * (1 + pre.double().abs()) if act != "none" else torch.zeros((), dtype=torch.float64, device=DEV)
    g, e = dy.double() * s, dy.double().abs() * es
    e = e + U * (g.abs() + e)
    assert ((dpre.double() - g).abs() <= e + BF * (g.abs() + e) + 2.0 ** -134).all()
    flat.check(f64(g.sum(0)), f64(e.sum(0) + (rows + 2) * U * (g.abs() + e).sum(0)), -0.5, 0, "bias")


@pytest.mark.parametrize("flags", FLAG_SETS)
@pytest.mark.parametrize("gaps", [False, True])
def test_bias_gradient_flags(flags, gaps):
    L, pl = odd_layout(300, gaps)
    dy = ints(1, 77, 300)
    flat = Flat(L, pl, 300, DEV, ints=True)
    z.zero_bias_grad(L, 1, dy, flat.acc, 0.5, flags, flat.out)
    flat.check(f64(dy.double().sum(0)), np.zeros(300), 0.5, flags, "bias")
    none = dy[:0]
    flat = Flat(L, pl, 300, DEV, ints=True)
    z.zero_bias_grad(L, 1, none, flat.acc, 0.5, flags, flat.out)
    flat.check(np.zeros(300), np.zeros(300), 0.5, flags, "no rows")


def test_nothing_to_do():
    w = Weights(8, 16, False)
    none = torch.empty(0, 16, dtype=BF16, device=DEV)
    z.zero_linear(w.L, 1, w.params, none, torch.empty(0, 8, dtype=BF16, device=DEV), bias=3, activation="gelu")
    z.zero_linear_input_grad(w.L, 1, w.params, torch.empty(0, 8, dtype=BF16, device=DEV), none)


@pytest.mark.parametrize("tr", [False, True])
def test_output_rows_past_32_bits(tr):
    """Rows of the result and of x that lie past 2^32 elements."""
    o, i, t = 24, 40, 300
    stride = 1 << 24
    w = Weights(o, i, tr, fill=lambda n: ints(n, n))
    big = torch.zeros(t * stride, dtype=BF16, device=DEV)          # 5.0e9 elements
    x = big.view(t, stride)[:, :i]
    x.copy_(ints(1, t, i))
    out = big.view(t, stride)[:, stride - o:]
    z.zero_linear(w.L, 1, w.params, x, torch.empty(t, o, dtype=F32, device=DEV), transposed=tr)
    exp = x.double() @ w.w.t()
    near = torch.empty(t, o, dtype=BF16, device=DEV)
    z.zero_linear(w.L, 1, w.params, x.contiguous(), near, transposed=tr)
    assert torch.equal(near, exp.float().bfloat16())
    far = torch.zeros(t * stride, dtype=BF16, device=DEV).view(t, stride)[:, :o]
    z.zero_linear(w.L, 1, w.params, x, far, transposed=tr)
    assert torch.equal(far, near) and not bool(out.any())


def test_captured_streams_and_workspaces():
    """Split sums and copied operands in two graphs replayed at once, with
    eager calls between, each replay checked."""
    t, o, i = 300, 264, 1030
    w = Weights(o, i, False, lead=17, fill=lambda n: ints(n, n))
    x, dy = ints(1, t, i), ints(2, t, o)
    exp = (x.double() @ w.w.t()).float(), (dy.double() @ w.w).float().bfloat16(), f64(dy.double().sum(0))
    side = torch.cuda.Stream()

    def calls(out, dx, acc, **kw):
        z.zero_linear(w.L, 1, w.params, x, out, **kw)
        z.zero_linear_input_grad(w.L, 1, w.params, dy, dx, **kw)
        z.zero_bias_grad(w.L, 3, dy, acc, 1.0, z.ACC_OVERWRITE, **kw)
    new = lambda: (torch.zeros(t, o, device=DEV), torch.zeros(t, i, dtype=BF16, device=DEV),  # noqa: E731
                   torch.zeros(w.L.padded, device=DEV))
    graphs = []
    for _ in range(2):
        bufs, g = new(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls(*bufs)
        graphs.append((g, bufs))
    at = int(w.L.tensor_flat(3)[0])
    for _ in range(4):
        for _, bufs in graphs:
            for b in bufs:
                b.zero_()
        for s, (g, _) in zip((side, torch.cuda.current_stream()), graphs):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        eager = new()
        torch.cuda.synchronize()
        calls(*eager, stream=side)
        torch.cuda.synchronize()
        for bufs in [b for _, b in graphs] + [eager]:
            assert torch.equal(bufs[0], exp[0]) and torch.equal(bufs[1], exp[1])
            assert np.array_equal(f64(bufs[2])[at:at + o], exp[2])


def test_the_same_bits_every_time():
    w = Weights(1000, 776, False)
    x = randn(1, 333, 776)
    outs = []
    for _ in range(3):
        outs.append(torch.empty(333, 1000, device=DEV))
        z.zero_linear(w.L, 1, w.params, x, outs[-1], bias=3, activation="silu")
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# Tiles of 256: of one block each, ragged; split over three blocks, with a sum of
# odd length; whole ones and the split rest of them.
LARGE = [(3000, 4160, 384), (3000, 384, 4160), (1000, 4160, 4100), (4100, 1000, 4104), (1000, 4104, 4160),
         (4100, 5000, 4100)]


@pytest.mark.parametrize("tr", [False, True])
@pytest.mark.parametrize("t,o,i", LARGE)
def test_large_tiles(t, o, i, tr):
    test_whole_numbers(t, o, i, tr)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("t,o,i,tr", [(3000, 4160, 384, False), (3001, 4160, 384, True), (1000, 4160, 4100, False),
                                      (1000, 4160, 4104, True)])
def test_large_tiles_epilogues(act, t, o, i, tr):
    test_epilogues(act, t, o, i, tr)


@pytest.mark.parametrize("tr", [False, True])
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("m,n,k", LARGE_TILES)
def test_sizes_of_large_tiles(m, n, k, grad, tr):
    """Each of these products, forward and as an input gradient, both orders of the weight."""
    test_whole_numbers(m, *((k, n) if grad else (n, k)), tr)


@pytest.mark.parametrize("act,tr", [("gelu", False), ("silu", True)])
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("m,n,k", [s for s in LARGE_TILES if s[0] % 2])
def test_epilogues_of_large_tiles(act, m, n, k, grad, tr):
    test_epilogues(act, m, *((k, n) if grad else (n, k)), tr)
