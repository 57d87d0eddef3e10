"""Plain references of the 8-bit moments: the format by its table of values,
rounding by the definition in 64 bits, and the step by the CPU oracle on the
values that the codes stand for."""
import numpy as np

import oracle
from micrograd_ref import E4M3, act8

V8 = np.array([c * 2.0 ** -18 if c < 16 else (1 + (c & 15) / 16) * 2.0 ** ((c >> 4) - 15)
               for c in range(255)])
KINDS = ("m", "v")


def random_bits(seed, t, i):
    """The 32 bits of the elements i (int64 array), in Python's whole numbers."""
    m64, m32 = (1 << 64) - 1, np.uint64((1 << 32) - 1)
    x = (seed ^ (t * 0x9E3779B97F4A7C15)) & m64
    for _ in range(2):
        x = ((x ^ (x >> 32)) * 0xD6E8FEB86659FD93) & m64
    x ^= x >> 32
    k0, k1 = np.uint64(x & 0xFFFFFFFF), np.uint64(x >> 32)
    i = np.asarray(i, np.int64).astype(np.uint64)
    u = np.uint64
    h = ((i & m32) * u(0x9E3779B1) + (i >> u(32)) * u(0x85EBCA77) + k0) & m32
    h = ((h ^ (h >> u(16))) * u(0xC2B2AE3D) + k1) & m32
    h = ((h ^ (h >> u(15))) * u(0x27D4EB2F)) & m32
    return h ^ (h >> u(16))


def scale_byte(kind, blk):
    mag = np.abs(blk[np.isfinite(blk)]).max(initial=0)
    if mag == 0:
        return 10 if kind == "m" else 19
    m, k = np.frexp(mag)                       # mag = 2m * 2^(k-1)
    if kind == "m":
        return max(10, 127 + (int(k) - 1) - 8 + (2 * m > 1.75))
    return min(253, max(19, 127 + int(k) - 1 + (2 * m > 1.875)))


def encode(kind, x, r=None):
    """(codes, scale bytes) of one slice of float32 values; r: 16 random bits
    an element, None for the nearest code."""
    x = np.asarray(x, np.float64)
    codes = np.zeros(x.size, np.uint8)
    scales = np.zeros(-(-x.size // 128), np.uint8)
    table = E4M3 if kind == "m" else V8
    first = 2.0 ** -6 if kind == "m" else 2.0 ** -14          # the smallest normal code's value
    frac = 3 if kind == "m" else 4
    grain = first * 2.0 ** -23
    for b in range(scales.size):
        at = slice(b * 128, (b + 1) * 128)
        blk = x[at]
        e = scale_byte(kind, blk)
        scales[b] = e
        fin = np.isfinite(blk)
        v = np.abs(np.where(fin, blk, 0)) / 2.0 ** (e - 127)
        v = np.where(v < first, np.round(v / grain) * grain, v)
        ex = np.floor(np.log2(np.maximum(v, first)))
        ex = np.where(2.0 ** ex > v, ex - 1, np.where(2.0 ** (ex + 1) <= v, ex + 1, ex))
        step = np.maximum(2.0 ** ex, first) * 2.0 ** -frac
        if r is None:
            q = np.round(v / step) * step                     # ties to even: a code's last bit is its step's
        else:
            q = np.floor(v / step + (r[at].astype(np.float64) + 0.5) / 65536) * step
        q = np.minimum(q, table[-1])
        c = np.searchsorted(table, q)
        assert np.array_equal(table[c], q)
        if kind == "m":
            c = np.where(fin, c, 0x7F) | np.where(np.signbit(blk), 0x80, 0)
        else:
            c = np.where(fin, np.maximum(c, blk > 0), 0xFF)
        codes[at] = c
    return codes, scales


def decode(kind, codes, scales):
    table = np.append(E4M3, np.nan) if kind == "m" else np.append(V8, np.nan)
    v = table[codes & 0x7F] if kind == "m" else table[codes]
    if kind == "m":
        v = np.where(codes & 0x80, -v, v)
    s = np.exp2(scales.astype(np.float64) - 127)
    return (v * np.repeat(s, 128)[:codes.size]).astype(np.float32)


def slices(pl):
    """(first element, elements, first scale byte) of every bucket's slice."""
    out, s = [], 0
    for off, padded in zip(pl.shard_off, pl.padded_len):
        n = int(padded) // pl.n_d
        out.append((int(off), n, s))
        s += -(-n // 128)
    return out, s


def each(pl, f):
    """f(first, elements, first scale byte, scale bytes) over the slices that hold anything."""
    for off, n, s in slices(pl)[0]:
        if n:
            f(off, n, s, -(-n // 128))


def decode_shard(kind, pl, codes, scales):
    out = np.zeros(codes.size, np.float32)

    def one(off, n, s, k):
        out[off:off + n] = decode(kind, codes[off:off + n], scales[s:s + k])
    each(pl, one)
    return out


def encode_shard(kind, pl, x, r=None):
    codes, scales = np.zeros(x.size, np.uint8), np.zeros(slices(pl)[1], np.uint8)

    def one(off, n, s, k):
        codes[off:off + n], scales[s:s + k] = encode(kind, x[off:off + n], None if r is None else r[off:off + n])
    each(pl, one)
    return codes, scales


def step(pl, grads, master, state, hp, t, seed):
    """The step on numpy arrays: bf16 patterns (uint16) or float32
    contributions in shard order; state: {"m": (codes, scales), "v": ...}.
    -> (master, bf16 patterns, new state)."""
    th = master.copy()
    m, v = (decode_shard(k, pl, *state[k]) for k in KINDS)
    run = oracle.shard_step if grads[0].dtype == np.uint16 else oracle.shard_step_f32
    with np.errstate(all="ignore"):
        p, _ = run(grads, th, m, v, hp, t)
    h = random_bits(seed, t, np.arange(th.size))
    return th, p, {"m": encode_shard("m", pl, m, h & np.uint64(0xFFFF)),
                   "v": encode_shard("v", pl, v, h >> np.uint64(16))}


def check_against_act8():
    """The first moment's nearest codes are the 8-bit activations'."""
    x = np.random.default_rng(0).normal(size=300).astype(np.float32)
    a, b = encode("m", x), act8(x[None])
    return np.array_equal(a[0], b[0][0]) and np.array_equal(a[1], b[1][0])
