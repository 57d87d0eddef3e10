"""Plain 64-bit references of the micro-batch operators (embedding, norm,
8-bit activations, weight gradient), and layouts to run them in.

U is half a step of binary32, BF that of bf16: what one rounding can be off,
relative to the value.
"""
import numpy as np
import torch

import fsdp_sharded_optimizer_step_amd as z
import oracle

U, BF = 2.0 ** -24, 2.0 ** -8

# values of the 128 non-negative e4m3 codes; 0x7f is NaN
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7)
                 for c in range(127)])


def layout(numel, gaps, n_d=4, dim0_rows=None):
    """A layout in which tensor 1 has `numel` elements at an odd offset.
    gaps: buckets of a length that n_d does not divide cut the tensor, so
    padding falls inside it."""
    sizes = [17, numel, 5]
    if dim0_rows is not None:
        return z.Layout(sizes, 0, n_d, 1, rows=[17, dim0_rows, 5]), oracle.plan(
            sizes, 0, n_d, rows=[17, dim0_rows, 5])
    cap = 0 if not gaps else max(3, numel // 3 // n_d * n_d + 1)
    return z.Layout(sizes, cap, n_d, 1), oracle.plan(sizes, cap, n_d)


def positions(pl, numel):
    """Flat position of every element of tensor 1."""
    x = 17 + np.arange(numel, dtype=np.int64)
    b = np.searchsorted(pl.stream_off, x, side="right") - 1
    # empty buckets share an offset with the next one: take the one that holds x
    return np.asarray(pl.padded_off)[b] + (x - np.asarray(pl.stream_off)[b])


def act8(x):
    """(codes, bytes) of the rows of x (float64 values of the input type)."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    nb = -(-cols // 128)
    codes = np.zeros((rows, cols), np.uint8)
    scales = np.zeros((rows, nb), np.uint8)
    for b in range(nb):
        blk = x[:, b * 128:(b + 1) * 128]
        mag = np.where(np.isfinite(blk), np.abs(blk), 0).max(1, initial=0)
        m, k = np.frexp(mag)                       # mag = 2m * 2^(k-1)
        e = np.where(mag > 0, 127 + (k - 1) - 8 + (2 * m > 1.75), 10)
        e = np.maximum(10, e)
        scales[:, b] = e
        with np.errstate(invalid="ignore"):
            v = np.abs(blk) / np.exp2(e - 127.0)[:, None]
        hi = np.clip(np.searchsorted(E4M3, np.where(np.isfinite(v), v, 0)), 1, 126)
        lo = hi - 1
        dl, dh = np.where(np.isfinite(v), v, 0) - E4M3[lo], E4M3[hi] - np.where(np.isfinite(v), v, 0)
        c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
        c = np.where(np.isfinite(v), c | np.where(np.signbit(blk), 0x80, 0), 0x7F)
        codes[:, b * 128:(b + 1) * 128] = c
    return codes, scales


def act8_values(codes, scales):
    v = np.append(E4M3, np.nan)[codes & 0x7F]
    v = np.where(codes & 0x80, -v, v)
    s = np.exp2(scales.astype(np.float64) - 127)
    return v * np.repeat(s, 128, axis=1)[:, :codes.shape[1]]


def f64(t):
    """A tensor's values; 16-bit integer tensors hold bf16 patterns."""
    if t.dtype in (torch.int16, torch.uint16):
        t = t.view(torch.bfloat16)
    return t.detach().cpu().double().numpy()


def apply_grad(acc, g, scale, flags):
    """(accumulator, emitted value) in 64 bits; None where not written."""
    a = scale * g + (0 if flags & z.ACC_OVERWRITE else acc)
    return (None if flags & z.ACC_NO_STORE else a), (a if flags & z.ACC_EMIT_BF16 else None)


FLAG_SETS = [0, z.ACC_OVERWRITE, z.ACC_EMIT_BF16, z.ACC_EMIT_BF16 | z.ACC_NO_STORE,
             z.ACC_OVERWRITE | z.ACC_EMIT_BF16 | z.ACC_NO_STORE,
             z.ACC_OVERWRITE | z.ACC_EMIT_BF16]


class Flat:
    """Accumulator and bf16 buffer of a layout, filled with known values, and
    the check of what a call left in them."""

    def __init__(self, L, pl, numel, dev, seed=0, ints=False):
        g = torch.Generator().manual_seed(seed)
        self.pos = positions(pl, numel)
        acc = torch.randint(-9, 10, (L.padded,), generator=g).float() if ints else \
            torch.randn(L.padded, generator=g)
        self.acc0 = acc.double().numpy().copy()
        self.acc = acc.to(dev)
        self.out = torch.full((L.padded,), 3.0, dtype=torch.bfloat16, device=dev)

    def check(self, g, bound, scale, flags, what):
        """g: exact gradient; bound: how far the kernel's sum may be off."""
        acc, out = f64(self.acc), f64(self.out)
        a0 = self.acc0[self.pos]
        a, e = apply_grad(a0, g, scale, flags)
        # product and sum round once each
        prod = np.abs(scale) * (np.abs(g) + bound)
        off = np.abs(scale) * bound + U * prod + U * (prod + np.abs(a0)) * (1 + U)
        rest = np.ones(acc.size, bool)
        rest[self.pos] = False
        assert np.array_equal(acc[rest], self.acc0[rest]), f"{what}: accumulator outside the tensor"
        assert (out[rest] == 3.0).all(), f"{what}: bf16 buffer outside the tensor"
        exp = a0 if a is None else a
        d = np.abs(acc[self.pos] - exp)
        assert (d <= (0 if a is None else off)).all(), \
            f"{what}: accumulator off by {np.max(d - off)} over the bound at {np.argmax(d - off)}"
        if e is None:
            assert (out[self.pos] == 3.0).all(), f"{what}: bf16 buffer written"
        else:
            d = np.abs(out[self.pos] - e)
            lim = off + BF * (np.abs(e) + off) + 2.0 ** -134
            assert (d <= lim).all(), f"{what}: emitted values off by {np.max(d - lim)}"
