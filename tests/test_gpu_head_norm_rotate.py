"""Norm of query and key heads and their rotation on the GPU, both directions,
against 64-bit references.

Tolerances.  U = 2^-24 is half a step of binary32, BF = 2^-8 of bf16.  A row's
sum of d squares is off by (d + 1) U of itself, 1/rms by half of that and four
roundings; a cosine or sine by T = 2^-20 (its angle, in turns of at most 1/2,
is rounded once to binary32, 2 pi 2^-26 at most, and the function gives 2
units of the last place) plus 2^-50 of the angle (the product in 64 bits).
"""
import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_step_amd as z
from micrograd_ref import BF, FLAG_SETS, U, Flat, f64, layout, positions
from test_gpu_micrograd import randn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16
T0 = 2.0 ** -20


@pytest.fixture(autouse=True)
def _free_gpu_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def pairs_of(half, inter):
    j = np.arange(half)
    return (2 * j, 2 * j + 1) if inter else (j, half + j)


def angles(rot):
    if rot is None:
        return np.zeros((1, 0))
    p = np.atleast_2d(rot.positions.cpu().numpy()).astype(np.float64)
    sec = rot.sections if rot.sections is not None else [rot.freqs.numel()]
    axis = np.repeat(np.arange(len(sec)), sec)
    return p[axis].T * rot.freqs.cpu().numpy()              # (tokens, pairs)


def turned(x, rot, sign):
    """(rows turned, bound on what the angles' errors and the products' roundings do)."""
    a = angles(rot)[:, None, :]
    i, j = pairs_of(a.shape[2], rot is not None and rot.interleaved)
    y, off = x.copy(), np.zeros_like(x)
    c, s = np.cos(a), sign * np.sin(a)
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., i] * s + x[..., j] * c
    mag = np.abs(x[..., i]) + np.abs(x[..., j])
    off[..., i] = off[..., j] = mag * (T0 + 2.0 ** -50 * np.abs(a) + 3 * U)
    return y, off


def forward(x, w, rot, eps):
    """(values, bound) of rows (tokens, heads, d)."""
    d = x.shape[2]
    if w is None:
        u, rel = x, 0.0
    else:
        u, rel = x / np.sqrt((x * x).mean(2, keepdims=True) + eps) * w, (d / 2 + 8) * U
    y, off = turned(u, rot, 1)
    a = angles(rot)
    i, j = pairs_of(a.shape[1], rot is not None and rot.interleaved)
    both = np.abs(u).copy()
    both[..., i] = both[..., j] = np.abs(u[..., i]) + np.abs(u[..., j])
    off = off + rel * both
    return y, off + BF * (np.abs(y) + off) + 2.0 ** -134


def backward(dy, x, w, rot, eps):
    """(dx, its bound, weight gradient, its bound)."""
    u, eu = turned(dy, rot, -1)
    if w is None:
        return u, eu + BF * (np.abs(u) + eu) + 2.0 ** -134, None, None
    d = x.shape[2]
    R = 1 / np.sqrt((x * x).mean(2, keepdims=True) + eps)
    n, g = x * R, u * w
    rel = (d / 2 + 10) * U
    dx = R * (g - n * (g * n).mean(2, keepdims=True))
    N, G = np.abs(n), np.abs(g)
    mean = (G * N).mean(2, keepdims=True)
    off = R * (eu * np.abs(w) + G * rel + N * ((eu * np.abs(w) * N).mean(2, keepdims=True) + mean * (2 * d + 24) * U))
    rows = x.shape[0] * x.shape[1]
    dw = (u * n).sum((0, 1))
    odw = (eu * N).sum((0, 1)) + (rows + d / 2 + 12) * U * (np.abs(u) * N).sum((0, 1))
    return dx, off + BF * (np.abs(dx) + off) + 2.0 ** -134, dw, odw


def rotation(t, half, axes=1, inter=False, start=0, seed=0, dtype=torch.int32, theta=10000.0):
    if half == 0:
        return None
    g = torch.Generator().manual_seed(seed)
    p = [torch.arange(t) + start] + [torch.randint(-50, 50, (t,), generator=g) for _ in range(axes - 1)]
    cut = [half // axes + (1 if a < half % axes else 0) for a in range(axes)]
    f = theta ** (-torch.arange(half, dtype=torch.float64) / half)
    p = torch.stack(p).to(dtype).to(DEV)
    return z.Rotation(p if axes > 1 else p[0], f.to(DEV), cut if axes > 1 else None, inter)


def close(got, exp, bound, what):
    d = np.abs(f64(got) - exp)
    assert (d <= bound).all(), f"{what}: off by {np.max(d - bound)} over the bound at {np.unravel_index(np.argmax(d - bound), d.shape)}"


CASES = [  # tokens, query heads, key heads, columns, turning columns, axes, interleaved
    (1, 1, 1, 2, 2, 1, False), (1, 32, 8, 128, 128, 1, False), (3, 2, 1, 1, 0, 1, False),
    (5, 3, 2, 8, 8, 1, True), (7, 4, 4, 16, 16, 1, False), (33, 5, 1, 24, 16, 1, False),
    (65, 2, 2, 64, 64, 3, True), (65, 2, 2, 64, 64, 3, False), (40, 3, 1, 80, 32, 2, False),
    (40, 3, 1, 80, 80, 4, True), (19, 12, 12, 96, 96, 1, False), (19, 2, 7, 100, 50, 1, False),
    (10, 1, 2, 33, 32, 1, True), (10, 2, 1, 77, 18, 2, False), (9, 8, 1, 192, 64, 1, True),
    (130, 4, 2, 256, 256, 1, False), (6, 3, 3, 257, 256, 3, False), (12, 2, 1, 512, 512, 1, False),
    (12, 2, 1, 504, 500, 1, True), (300, 17, 5, 128, 64, 1, False), (4, 2, 2, 128, 0, 1, False),
    (2000, 3, 1, 64, 64, 1, False), (1, 2, 0, 64, 64, 1, False), (1, 0, 3, 64, 64, 1, False)]


@pytest.mark.parametrize("normed", [True, False])
@pytest.mark.parametrize("t,hq,hk,d,r,axes,inter", CASES)
def test_both_directions(t, hq, hk, d, r, axes, inter, normed):
    L, pl = layout(d, False)
    params = randn(d, L.padded) * 0.2 + 1
    w = f64(params)[positions(pl, d)] if normed else None
    rot = rotation(t, r // 2, axes, inter, start=1000 * t, seed=d)
    eps = 1e-5
    x = [randn(1 + n, t, h, d, scale=3.0) for n, h in ((0, hq), (1, hk))]
    x[0][0, :1] = 0                                        # a row of zeros
    dy = [randn(5 + n, t, h, d) for n, h in ((0, hq), (1, hk))]
    out = [torch.full_like(a, 9) for a in x]
    use = lambda v: [a if h else None for a, h in zip(v, (hq, hk))]  # noqa: E731
    tensor = 1 if normed else None
    z.zero_head_norm_rotate(L, tensor, tensor, params, *use(x), eps, rot, *use(out))
    for a, o, n in zip(x, out, "qk"):
        close(o, *forward(f64(a), w, rot, eps), n)
    flat = Flat(L, pl, d, DEV, seed=t)
    dx = [torch.full_like(a, 9) for a in x]
    z.zero_head_norm_rotate_grad(L, tensor, tensor, params, *use(dy), *use(x), eps, rot, *use(dx), flat.acc, 0.25)
    dw, odw = np.zeros(d), np.zeros(d)
    for a, b, o, n in zip(dy, x, dx, "qk"):
        g, bound, s, os_ = backward(f64(a), f64(b), w, rot, eps)
        close(o, g, bound, n + " gradient")
        if normed:
            dw, odw = dw + s, odw + os_
    # the two sides' sums are added up
    flat.check(dw if normed else np.zeros(d), odw + U * np.abs(dw), 0.25 if normed else 0.0, 0, "weight")


@pytest.mark.parametrize("flags", FLAG_SETS)
@pytest.mark.parametrize("gaps,d,inter", [(False, 64, False), (True, 64, False), (True, 90, True)])
def test_weights_of_their_own_and_flags(flags, gaps, d, inter):
    """Queries' and keys' weights are different tensors, with bucket padding inside."""
    import oracle
    sizes, n_d = [5, d, 3, d], 4
    cap = d // 3 // n_d * n_d + 1 if gaps else 0
    L, pl = z.Layout(sizes, cap, n_d, 0), oracle.plan(sizes, cap, n_d)

    def place(first):
        x = first + np.arange(d)
        b = np.searchsorted(pl.stream_off, x, side="right") - 1
        return np.asarray(pl.padded_off)[b] + x - np.asarray(pl.stream_off)[b]
    at = [place(5), place(5 + d + 3)]
    params = randn(1, L.padded) + 1
    w = [f64(params)[p] for p in at]
    t, heads = 50, (6, 2)
    rot = rotation(t, 16, 1, inter)
    x = [randn(2 + n, t, h, d) for n, h in enumerate(heads)]
    dy = [randn(4 + n, t, h, d) for n, h in enumerate(heads)]
    out, dx = [torch.empty_like(a) for a in x], [torch.empty_like(a) for a in x]
    z.zero_head_norm_rotate(L, 1, 3, params, *x, 1e-6, rot, *out)
    acc, emit = torch.randn(L.padded, device=DEV), torch.full((L.padded,), 3.0, dtype=BF16, device=DEV)
    a0 = f64(acc)
    z.zero_head_norm_rotate_grad(L, 1, 3, params, *dy, *x, 1e-6, rot, *dx, acc, -0.5, flags, emit)
    rest = np.ones(L.padded, bool)
    for n in range(2):
        close(out[n], *forward(f64(x[n]), w[n], rot, 1e-6), "out")
        g, bound, s, os_ = backward(f64(dy[n]), f64(x[n]), w[n], rot, 1e-6)
        close(dx[n], g, bound, "gradient")
        flat = Flat.__new__(Flat)
        flat.pos, flat.acc0, rest[at[n]] = at[n], a0, False
        flat.acc, flat.out = acc.clone(), emit.clone()
        other = at[1 - n]
        flat.acc[other], flat.out[other] = torch.from_numpy(a0[other]).float().to(DEV), 3.0
        flat.check(s, os_, -0.5, flags, "weight %d" % n)
    assert np.array_equal(f64(acc)[rest], a0[rest]) and (f64(emit)[rest] == 3).all()


@pytest.mark.parametrize("d,r", [(128, 128), (96, 32), (50, 48)])
def test_views_of_one_projection_and_heads_in_front(d, r):
    """Queries, keys and values of a token in one row, of odd length and start;
    outputs that take turns in one buffer; outputs with the heads in front."""
    t, hq, hk = 37, 6, 2
    L, pl = layout(d, False)
    params = randn(d, L.padded) + 1
    w = f64(params)[positions(pl, d)]
    rot = rotation(t, r // 2)
    width = (hq + 2 * hk) * d
    qkv = randn(3, t * (width + 3) + 1)[1:].view(t, width + 3)
    q, k = qkv[:, :hq * d].view(t, hq, d), qkv[:, hq * d:(hq + hk) * d].view(t, hk, d)
    exp = [forward(f64(a), w, rot, 1e-6) for a in (q, k)]
    both = torch.full((t, hq + hk + 1, d), 9, dtype=BF16, device=DEV)
    z.zero_head_norm_rotate(L, 1, 1, params, q, k, 1e-6, rot, both[:, :hq], both[:, hq:hq + hk])
    close(both[:, :hq], *exp[0], "q")
    close(both[:, hq:hq + hk], *exp[1], "k")
    assert (both[:, -1] == 9).all()
    front = torch.full((hq + hk, t, d), 9, dtype=BF16, device=DEV)
    z.zero_head_norm_rotate(L, 1, 1, params, q, k, 1e-6, rot, front[:hq].transpose(0, 1), front[hq:].transpose(0, 1))
    assert torch.equal(front.transpose(0, 1), both[:, :-1])
    # the gradient into a buffer laid out like the projection's output
    dy = randn(4, t, hq + hk, d)
    dqkv = torch.full((t, width), 9, dtype=BF16, device=DEV)
    acc = torch.zeros(L.padded, device=DEV)
    views = [dqkv[:, :hq * d].view(t, hq, d), dqkv[:, hq * d:(hq + hk) * d].view(t, hk, d)]
    z.zero_head_norm_rotate_grad(L, 1, 1, params, dy[:, :hq], dy[:, hq:], q, k, 1e-6, rot, *views, acc)
    for v, a, x, n in zip(views, (dy[:, :hq], dy[:, hq:]), (q, k), "qk"):
        close(v, *backward(f64(a), f64(x), w, rot, 1e-6)[:2], n)
    assert (dqkv[:, (hq + hk) * d:] == 9).all()


@pytest.mark.parametrize("dtype,start", [(torch.int32, 2 ** 31 - 70), (torch.int64, 2 ** 31), (torch.int64, 10 ** 7),
                                         (torch.int32, -2 ** 31), (torch.int32, 131072)])
def test_far_positions(dtype, start):
    t, d = 64, 64
    L, _ = layout(d, False)
    rot = rotation(t, 32, start=start, dtype=dtype, theta=500000.0)
    x = randn(1, t, 3, d)
    out = torch.empty_like(x)
    z.zero_head_norm_rotate(L, None, None, None, x, None, 0.0, rot, out, None)
    close(out, *forward(f64(x), None, rot, 0), "out")


def test_rows_of_infinities_leave_the_others_alone():
    t, d = 9, 128
    L, _ = layout(d, False)
    params, rot = randn(d, L.padded), rotation(9, 64)
    x, dy = randn(1, t, 4, d), randn(2, t, 4, d)
    clean, acc = [torch.empty_like(x) for _ in range(2)], torch.zeros(L.padded, device=DEV)
    z.zero_head_norm_rotate(L, 1, None, params, x, None, 1e-6, rot, clean[0], None)
    z.zero_head_norm_rotate_grad(L, 1, None, params, dy, None, x, None, 1e-6, rot, clean[1], None, acc)
    bad = x.clone()
    bad[2, 1, 3], bad[4, 0, 0], bad[5, 3, 127] = float("inf"), float("nan"), float("-inf")
    out = [torch.empty_like(x) for _ in range(2)]
    z.zero_head_norm_rotate(L, 1, None, params, bad, None, 1e-6, rot, out[0], None)
    z.zero_head_norm_rotate_grad(L, 1, None, params, dy, None, bad, None, 1e-6, rot, out[1], None, acc)
    hit = torch.zeros(t, 4, dtype=torch.bool, device=DEV)
    hit[2, 1] = hit[4, 0] = hit[5, 3] = True
    for a, b in zip(clean, out):
        assert torch.equal(a[~hit], b[~hit])


@pytest.mark.parametrize("d,r,inter,top", [(128, 128, False, 1.5e19), (512, 512, True, 1.5e19), (100, 90, False, 1.5e19),
                                           (64, 64, True, 1.5e19), (128, 64, False, 4e18), (16, 16, False, 1e19),
                                           (512, 0, False, 1e-15), (512, 0, False, 2e-18), (100, 90, True, 2e-18)])
def test_rows_up_to_the_largest_mean_square(d, r, inter, top):
    """mean(x^2) up to 2.3e38, where the sum of the squares would be infinite, and
    down to 2e-36, where a part of the mean, 2^-127, is off by 2^-23 of itself."""
    t, h = 5, 3
    L, pl = layout(d, False)
    params, rot = randn(d, L.padded) + 1, rotation(t, r // 2, inter=inter)
    w = f64(params)[positions(pl, d)]
    x, dy = (randn(1, t, h, d).clamp(-1, 1) * top).to(BF16), randn(2, t, h, d)
    x[0, 0] = top                                          # every column
    out, dx, flat = torch.empty_like(x), torch.empty_like(x), Flat(L, pl, d, DEV)
    z.zero_head_norm_rotate(L, 1, None, params, x, None, 0.0, rot, out, None)
    close(out, *forward(f64(x), w, rot, 0.0), "out")
    dy *= 1e18 if top > 1 else 1e-15                       # mean(|g x|) stays below 3e38
    z.zero_head_norm_rotate_grad(L, 1, None, params, dy, None, x, None, 0.0, rot, dx, None, flat.acc, 2.0 ** -60)
    g, bound, dw, odw = backward(f64(dy), f64(x), w, rot, 0.0)
    close(dx, g, bound, "gradient")
    flat.check(dw, odw + U * np.abs(dw), 2.0 ** -60, 0, "weight")


def test_an_eps_too_small_for_binary32_keeps_rows_of_zeros():
    t, d = 5, 64
    L, _ = layout(d, False)
    params, rot = randn(d, L.padded) + 1, rotation(t, 32)
    x = randn(1, t, 2, d)
    x[1] = 0
    out = [torch.full_like(x, 9) for _ in range(3)]
    for o, eps in zip(out, (1e-60, 2.0 ** -149, 1e-300)):
        z.zero_head_norm_rotate(L, 1, None, params, x, None, eps, rot, o, None)
    assert not out[0][1].any() and torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])


@pytest.mark.parametrize("d,r,inter", [(128, 64, False), (128, 0, False), (128, 64, True), (64, 16, False),
                                       (96, 24, False), (80, 20, True), (33, 32, False), (7, 0, False)])
def test_columns_that_do_not_turn_leave_each_other_alone(d, r, inter):
    """An infinity or a NaN in one of them reaches no other column: without a
    norm they come out as they went in, in both directions."""
    t, h = 6, 3
    L, _ = layout(d, False)
    rot = rotation(t, r // 2, inter=inter)
    x = randn(1, t, h, d)
    new = lambda: [torch.empty_like(x) for _ in range(2)]  # noqa: E731

    def both(a, out):
        z.zero_head_norm_rotate(L, None, None, None, a, None, 0.0, rot, out[0], None)
        z.zero_head_norm_rotate_grad(L, None, None, None, a, None, None, None, 0.0, rot, out[1], None)
    clean, got, bad = new(), new(), x.clone()
    both(x, clean)
    for k, c in enumerate(range(r, d)):                     # every column once, in a row of its own if there are enough
        bad.view(t * h, d)[k % (t * h), c] = (float("inf"), float("nan"), float("-inf"))[k % 3]
    both(bad, got)
    hit = bad != x
    for a, b in zip(clean, got):
        assert torch.equal(a[~hit], b[~hit])
        assert torch.equal(torch.nan_to_num(b[hit].float(), 5.0), torch.nan_to_num(bad[hit].float(), 5.0))
        assert torch.equal(a[..., r:], x[..., r:])


def test_gradient_against_differences():
    """Sums of dy * out change along a direction by the gradient's product with
    it: central differences in 64 bits of the reference's forward pass against
    the kernel's gradients, whose own error is bounded as above."""
    t, h, d = 6, 3, 48
    L, pl = layout(d, False)
    params, rot = randn(d, L.padded) + 1, rotation(t, 16, 2, True)
    x, dy = randn(1, t, h, d), randn(2, t, h, d)
    w = f64(params)[positions(pl, d)]
    dx, acc = torch.empty_like(x), torch.zeros(L.padded, device=DEV)
    z.zero_head_norm_rotate_grad(L, 1, None, params, dy, None, x, None, 1e-6, rot, dx, None, acc)
    g = np.random.default_rng(0)
    vx, vw, step = g.normal(size=x.shape), g.normal(size=d), 1e-6
    loss = lambda s: (f64(dy) * forward(f64(x) + s * vx, w + s * vw, rot, 1e-6)[0]).sum()  # noqa: E731
    slope = (loss(step) - loss(-step)) / (2 * step)
    _, bx, _, bw = backward(f64(dy), f64(x), w, rot, 1e-6)
    got = (f64(dx) * vx).sum() + (f64(acc)[positions(pl, d)] * vw).sum()
    # the difference's own error: third derivatives times step^2, and 2^-52 of the loss over the step
    own = 1e-6 * np.abs(f64(dy) * x.shape[2]).sum()
    assert abs(got - slope) <= (bx * np.abs(vx)).sum() + ((bw + 2 * U * np.abs(f64(acc)).max()) * np.abs(vw)).sum() + own


@pytest.mark.parametrize("t,hq,hk", [(1, 3, 1), (5, 1, 1), (7, 2, 0), (13, 9, 5)])
def test_lanes_without_a_row_count_for_nothing(t, hq, hk):
    """Tokens and heads that do not fill a wave: with eps = 0 a row of zeros has
    no norm, and LDS may hold NaN from an earlier kernel."""
    d = 64
    L, pl = layout(d, False)
    params, rot = randn(d, L.padded) + 1, rotation(t, 32)
    w = f64(params)[positions(pl, d)]
    n = 1024
    W = z.Layout([n * n], 0, 1, 0)
    nan = torch.full((16 * n, n), float("nan"), dtype=BF16, device=DEV)
    z.zero_linear(W, 0, nan[:n].view(-1), nan, torch.empty_like(nan))
    x = [randn(1 + k, t, h, d) for k, h in enumerate((hq, hk))]
    dy = [randn(3 + k, t, h, d) for k, h in enumerate((hq, hk))]
    dx = [torch.empty_like(a) for a in x]
    use = lambda v: [a if h else None for a, h in zip(v, (hq, hk))]  # noqa: E731
    flat = Flat(L, pl, d, DEV)
    z.zero_head_norm_rotate_grad(L, 1, 1, params, *use(dy), *use(x), 0.0, rot, *use(dx), flat.acc)
    dw, odw = np.zeros(d), np.zeros(d)
    for a, b, o in zip(dy, x, dx):
        if a.shape[1]:
            g, bound, s, os_ = backward(f64(a), f64(b), w, rot, 0.0)
            close(o, g, bound, "gradient")
            dw, odw = dw + s, odw + os_
    flat.check(dw, odw + U * np.abs(dw), 1.0, 0, "weight")


@pytest.mark.parametrize("flags", [0, z.ACC_OVERWRITE, z.ACC_EMIT_BF16])
def test_no_tokens(flags):
    L, pl = layout(64, False)
    none = torch.empty(0, 4, 64, dtype=BF16, device=DEV)
    rot = rotation(0, 32)
    params = randn(1, L.padded)
    z.zero_head_norm_rotate(L, 1, 1, params, none, none, 1e-6, rot, none, none)
    flat = Flat(L, pl, 64, DEV)
    z.zero_head_norm_rotate_grad(L, 1, 1, params, none, none, none, none, 1e-6, rot, none, none, flat.acc, 0.5,
                                 flags, flat.out)
    flat.check(np.zeros(64), np.zeros(64), 0.5, flags, "no tokens")


def test_offsets_beyond_32_bits():
    """Head strides that take an operand past 2^32 elements."""
    t, h, d = 5, 3, 128
    L, _ = layout(d, False)
    params, rot = randn(d, L.padded), rotation(t, 64)
    far = torch.zeros(2 * (1 << 31) + t * d, dtype=BF16, device=DEV)
    x = far.as_strided((t, h, d), (d, 1 << 31, 1))
    x.copy_(randn(1, t, h, d))
    near, out = x.contiguous(), torch.empty(t, h, d, dtype=BF16, device=DEV)
    z.zero_head_norm_rotate(L, 1, None, params, near, None, 1e-6, rot, out, None)
    other = torch.zeros_like(far).as_strided((t, h, d), (d, 1 << 31, 1))
    z.zero_head_norm_rotate(L, 1, None, params, x, None, 1e-6, rot, other, None)
    assert torch.equal(out, other)


def test_captured_and_replayed():
    """A graph of both directions, replayed with eager work between, and an
    eager call on another stream with a workspace of its own."""
    t, hq, hk, d = 700, 8, 2, 128
    L, _ = layout(d, False)
    params, rot = randn(d, L.padded) + 1, rotation(t, 64)
    q, k, dq, dk = (randn(n, t, h, d) for n, h in ((1, hq), (2, hk), (3, hq), (4, hk)))
    new = lambda: [torch.empty_like(q), torch.empty_like(k)]  # noqa: E731
    eager, acc = (new(), new()), torch.zeros(L.padded, device=DEV)

    def both(out, grad, acc, **kw):
        z.zero_head_norm_rotate(L, 1, 1, params, q, k, 1e-6, rot, *out, **kw)
        z.zero_head_norm_rotate_grad(L, 1, 1, params, dq, dk, q, k, 1e-6, rot, *grad, acc, 1.0, z.ACC_OVERWRITE, **kw)
    both(*eager, acc)
    graphs = []
    for _ in range(2):
        got, gacc = (new(), new()), torch.zeros_like(acc)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            both(*got, gacc)
        graphs.append((g, got, gacc))
    side = torch.cuda.Stream()
    for _ in range(4):
        for g, got, gacc in graphs:
            for a in got[0] + got[1] + [gacc]:
                a.zero_()
        for s, (g, _, _) in zip((side, torch.cuda.current_stream()), graphs):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        more, macc = (new(), new()), torch.zeros_like(acc)
        torch.cuda.synchronize()
        both(*more, macc, stream=side)
        torch.cuda.synchronize()
        for got, gacc in [x[1:] for x in graphs] + [(more, macc)]:
            for a, b in zip(eager[0] + eager[1] + [acc], got[0] + got[1] + [gacc]):
                assert torch.equal(a, b)
