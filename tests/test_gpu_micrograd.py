"""The micro-batch operators (embedding, norm, 8-bit activations, weight
gradient) on the GPU against plain 64-bit references.

Tolerances count roundings: a binary32 sum of n terms in any order is off by
at most n*U times the sum of the terms' magnitudes (U = 2^-24, to first order;
the constants below leave room for the products' own roundings), a value
rounded to bf16 by 2^-8 of itself.  Where inputs are small integers every sum
is exact and the results have to be equal.
"""
import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_step_amd as z
import oracle
from micrograd_ref import (BF, E4M3, FLAG_SETS, U, Flat, act8, act8_values, f64, layout, positions)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32, F8, U8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.uint8


@pytest.fixture(autouse=True)
def _free_gpu_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def randn(seed, *shape, dtype=BF16, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).to(DEV)


def strided(t, extra, offset=0):
    """The same matrix with rows `extra` elements further apart, starting
    `offset` elements into its memory."""
    rows, cols = t.shape
    buf = torch.full((offset + rows * (cols + extra) + 8,), 7, dtype=t.dtype, device=t.device)
    v = buf[offset:offset + rows * (cols + extra)].view(rows, cols + extra)[:, :cols]
    v.copy_(t)
    return v


def codes_like(rows, cols):
    return (torch.full((rows, cols), 0x55, dtype=U8, device=DEV),
            torch.full((rows, -(-cols // 128)), 0x55, dtype=U8, device=DEV))


# ------------------------------------------------------------------ act8
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols,extra,offset", [
    (1, 1, 0, 0), (3, 8, 0, 0), (5, 127, 3, 1), (4, 128, 0, 0), (4, 129, 0, 0), (33, 257, 7, 3),
    (64, 770, 0, 0), (7, 4096, 8, 0), (1, 14336, 0, 0), (2000, 40, 1, 1)])
def test_act8_codes_and_values_are_exact(dtype, rows, cols, extra, offset):
    x = strided(randn(rows + cols, rows, cols, dtype=dtype, scale=3.0), extra, offset)
    x[:, ::11] *= 2.0 ** -7
    x[0, 0] = 0.0
    q, e = codes_like(rows, cols)
    z.zero_act8_pack(x, q, e)
    eq, ee = act8(f64(x))
    assert np.array_equal(e.cpu().numpy(), ee)
    assert np.array_equal(q.cpu().numpy(), eq)
    for out_dtype in (BF16, F32):
        out = strided(torch.zeros(rows, cols, dtype=out_dtype, device=DEV), extra, offset)
        z.zero_act8_unpack(q.view(F8), e, out)
        assert np.array_equal(f64(out), act8_values(eq, ee))
        base = out.as_strided((rows, cols + extra), (cols + extra, 1)) if extra else None
        if base is not None:
            assert (base[:-1, cols:] == 7).all()


def test_act8_every_bf16_value():
    """Every bf16 pattern in a block of its own, and every one next to a value
    that fixes the scale at 1 (halfway cases, the smallest codes)."""
    pat = torch.arange(65536, dtype=torch.int32).to(torch.uint16).view(BF16)
    for x in (pat.view(-1, 1), torch.stack([torch.where(pat.abs() <= 448, pat, torch.zeros_like(pat)),
                                            torch.full_like(pat, 448.0)], 1)):
        x = x.contiguous().to(DEV)
        q, e = codes_like(*x.shape)
        z.zero_act8_pack(x, q, e)
        eq, ee = act8(f64(x))
        assert np.array_equal(e.cpu().numpy(), ee)
        got = q.cpu().numpy()
        nan = (eq & 0x7F) == 0x7F
        assert np.array_equal(nan, (got & 0x7F) == 0x7F)
        assert np.array_equal(got[~nan], eq[~nan])
        out = torch.empty_like(x)
        z.zero_act8_unpack(q, e, out)
        v, r = f64(out), act8_values(eq, ee)
        # magnitudes from 1.9375 * 2^127 round to the code 256 of the scale
        # 2^120: 2^128, which is past bf16's (and binary32's) largest value
        r = np.where(np.abs(r) == 2.0 ** 128, np.copysign(np.inf, r), r)
        assert np.array_equal(v[~nan], r[~nan]) and np.isnan(v[nan]).all()


def test_act8_non_finite_values_leave_their_block_alone():
    x = randn(1, 4, 300, dtype=F32)
    clean = x.clone()
    x[0, 5], x[1, 130], x[2, 299] = float("inf"), float("-inf"), float("nan")
    x[3, :128] = float("nan")
    clean[0, 5] = clean[1, 130] = clean[2, 299] = 0
    clean[3, :128] = 0
    q, e = codes_like(4, 300)
    z.zero_act8_pack(x, q, e)
    cq, ce = act8(f64(clean))
    bad = ~np.isfinite(f64(x))
    got = q.cpu().numpy()
    assert np.array_equal(e.cpu().numpy(), ce)
    assert ((got[bad] & 0x7F) == 0x7F).all() and np.array_equal(got[~bad], cq[~bad])


def test_act8_offsets_beyond_32_bits():
    rows, cols = 300_000, 14_400   # 4.3e9 codes
    x = torch.zeros(rows, cols, dtype=BF16, device=DEV)
    tail = randn(3, 2, cols)
    x[-2:] = tail
    q = torch.empty(rows, cols, dtype=U8, device=DEV)
    e = torch.empty(rows, -(-cols // 128), dtype=U8, device=DEV)
    z.zero_act8_pack(x, q, e)
    eq, ee = act8(f64(tail))
    assert np.array_equal(q[-2:].cpu().numpy(), eq) and np.array_equal(e[-2:].cpu().numpy(), ee)
    assert not q[rows - 3].any() and int(e[0, 0]) == 10
    x.fill_(9.0)
    z.zero_act8_unpack(q, e, x)
    assert np.array_equal(f64(x[-2:]), act8_values(eq, ee)) and not x[0].any()


# ------------------------------------------------------------------ lookup
@pytest.mark.parametrize("gaps", [False, True])
@pytest.mark.parametrize("id_dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("vocab,cols,n", [(7, 1, 1), (50, 8, 100), (33, 37, 65), (1000, 770, 17),
                                          (11, 4096, 300), (3, 8200, 5)])
def test_lookup(gaps, id_dtype, out_dtype, vocab, cols, n):
    L, pl = layout(vocab * cols, gaps)
    pos = positions(pl, vocab * cols)
    params = randn(vocab, L.padded)
    ids = torch.randint(-2, vocab + 2, (n,), generator=torch.Generator().manual_seed(n))
    ids[0] = vocab - 1
    out = strided(torch.zeros(n, cols, dtype=out_dtype, device=DEV), 3, 1)
    scale = cols ** 0.5
    z.zero_embedding_lookup(L, 1, params, ids.to(id_dtype).to(DEV), out, scale=scale)
    table = params.cpu()[torch.from_numpy(pos)].view(vocab, cols)
    real = (ids >= 0) & (ids < vocab)
    # one binary32 product, one rounding to the output: the same bits
    exp = table[ids.clamp(0, vocab - 1)].float() * torch.tensor(scale, dtype=F32)
    exp = torch.where(real[:, None], exp, torch.zeros(())).to(out_dtype)
    assert torch.equal(out.cpu(), exp)


def test_lookup_whole_rows_of_a_table_beyond_32_bits():
    vocab, cols = 300_001, 16_384   # 4.9e9 elements
    L = z.Layout([vocab * cols], 0, 8, 0)
    params = torch.zeros(L.padded, dtype=BF16, device=DEV)
    last = randn(5, cols)
    params[(vocab - 1) * cols:vocab * cols] = last
    out = torch.empty(3, cols, dtype=BF16, device=DEV)
    z.zero_embedding_lookup(L, 0, params, torch.tensor([vocab - 1, 5, vocab], device=DEV), out)
    assert torch.equal(out[0], last) and not out[1:].any()


# ------------------------------------------------------------------ embedding gradient
def emb_exact(ids, dy, vocab):
    g = np.zeros((vocab, dy.shape[1]))
    mag = np.zeros_like(g)
    cnt = np.zeros(vocab)
    real = (ids >= 0) & (ids < vocab)
    np.add.at(g, ids[real], dy[real])
    np.add.at(mag, ids[real], np.abs(dy[real]))
    np.add.at(cnt, ids[real], 1)
    return g.reshape(-1), (cnt[:, None] * U * mag).reshape(-1)


def some_ids(kind, n, vocab, seed=0):
    r = np.random.default_rng(seed)
    if kind == "uniform":
        return r.integers(0, vocab, n)
    if kind == "same":
        return np.full(n, vocab - 1)
    if kind == "skewed":
        return (vocab * r.random(n) ** 6).astype(np.int64)
    if kind == "holes":
        return r.integers(-vocab, 2 * vocab, n)
    return np.full(n, -1)               # "none"


@pytest.mark.parametrize("gaps", [False, True])
@pytest.mark.parametrize("flags", FLAG_SETS)
@pytest.mark.parametrize("kind", ["uniform", "skewed", "holes", "none"])
@pytest.mark.parametrize("n", [200, 700, 1024, 1025])
def test_emb_grad_flags(gaps, flags, kind, n):
    vocab, cols = 301, 37
    L, pl = layout(vocab * cols, gaps)
    ids = some_ids(kind, n, vocab)
    dy = strided(randn(2, n, cols), 5, 1)
    f = Flat(L, pl, vocab * cols, DEV)
    z.zero_embedding_grad(L, 1, torch.from_numpy(ids).to(DEV), dy, f.acc, 0.25, flags, f.out)
    f.check(*emb_exact(ids, f64(dy), vocab), 0.25, flags, f"{kind} {flags}")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("flags", [0, z.ACC_EMIT_BF16])
@pytest.mark.parametrize("vocab,cols,n,kind", [
    (1, 1, 1, "uniform"), (1, 5, 200, "same"), (5, 4, 63, "uniform"), (5, 4, 64, "same"),
    (5, 4, 65, "same"), (3, 130, 1000, "uniform"), (300_000, 3, 5000, "skewed"),
    (50257, 16, 3000, "skewed"), (100, 1000, 129, "same"), (1024, 64, 1, "uniform"),
    (257, 4100, 64, "holes"), (2, 8, 20000, "uniform"), (7, 1030, 512, "same"),
    (7, 1030, 513, "same"), (40, 2050, 512, "holes"), (40, 2050, 511, "skewed")])
def test_emb_grad_shapes_exact_in_integers(dtype, flags, vocab, cols, n, kind):
    """Small integers: every sum is exact, whatever its order."""
    L, pl = layout(vocab * cols, False)
    ids = some_ids(kind, n, vocab, n)
    dy = torch.from_numpy(np.random.default_rng(n).integers(-4, 5, (n, cols))).to(dtype).to(DEV)
    f = Flat(L, pl, vocab * cols, DEV, ints=True)
    z.zero_embedding_grad(L, 1, torch.from_numpy(ids.astype(np.int32)).to(DEV), dy, f.acc, 1.0,
                          flags, f.out)
    g, _ = emb_exact(ids, f64(dy), vocab)
    assert np.array_equal(f64(f.acc)[f.pos], f.acc0[f.pos] + g)
    f.acc0[f.pos] += g
    rest = np.setdiff1d(np.arange(L.padded), f.pos)
    assert np.array_equal(f64(f.acc)[rest], f.acc0[rest])


@pytest.mark.parametrize("gaps", [False, True])
@pytest.mark.parametrize("flags", FLAG_SETS)
@pytest.mark.parametrize("kind", ["skewed", "holes"])
def test_emb_grad_wide_rows(gaps, flags, kind):
    vocab, cols, n = 40, 2050, 1100
    L, pl = layout(vocab * cols, gaps)
    ids = some_ids(kind, n, vocab, 7)
    dy = strided(randn(2, n, cols), 3, 1)
    f = Flat(L, pl, vocab * cols, DEV)
    z.zero_embedding_grad(L, 1, torch.from_numpy(ids).to(DEV), dy, f.acc, 0.25, flags, f.out)
    f.check(*emb_exact(ids, f64(dy), vocab), 0.25, flags, f"{kind} {flags}")


# so many tokens that they are dealt to the slices first: one more than are
# not, chunks of 1024 and of more, a last chunk of one token, wide and narrow
# rows, ids of 1023 tokens and more
@pytest.mark.parametrize("id_dtype", [np.int32, np.int64])
@pytest.mark.parametrize("flags", [0, z.ACC_OVERWRITE | z.ACC_EMIT_BF16])
@pytest.mark.parametrize("vocab,cols,n,kind", [
    (50257, 3, 16384, "skewed"), (50257, 3, 16385, "skewed"), (300, 66, 20000, "same"),
    (1000, 130, 20000, "holes"), (262144, 2, 40961, "uniform"), (262145, 2, 40961, "uniform"),
    (2, 5, 300_000, "uniform"), (257, 1, 262_145, "skewed"), (17, 1030, 17000, "skewed"),
    (1, 261, 33000, "uniform"), (5000, 257, 17001, "same"), (1500, 8, 1151, "same"),
    (1500, 8, 1152, "same"), (3, 65, 1600, "holes"), (3, 1100, 2500, "uniform")])
def test_emb_grad_of_many_tokens_exact_in_integers(vocab, cols, n, kind, flags, id_dtype):
    L, pl = layout(vocab * cols, vocab * cols > 8 and n % 2 == 1)
    ids = some_ids(kind, n, vocab, n).astype(id_dtype)
    ids[::9] = np.array([-1, vocab, 0, np.iinfo(id_dtype).max], id_dtype)[np.arange(len(ids[::9])) % 4]
    dy = torch.from_numpy(np.random.default_rng(n).integers(-4, 5, (n, cols))).to(BF16).to(DEV)
    f = Flat(L, pl, vocab * cols, DEV, ints=True)
    z.zero_embedding_grad(L, 1, torch.from_numpy(ids).to(DEV), dy, f.acc, 1.0, flags, f.out)
    at = (ids >= 0) & (ids < vocab)
    g = np.zeros((vocab, cols))
    np.add.at(g, ids[at], f64(dy)[at])
    want = (0 if flags & z.ACC_OVERWRITE else f.acc0[f.pos]) + g.reshape(-1)
    assert np.array_equal(f64(f.acc)[f.pos], want)
    f.check(g.reshape(-1), np.zeros(g.size), 1.0, flags, kind)


@pytest.mark.parametrize("gaps", [False, True])
@pytest.mark.parametrize("flags", [0, z.ACC_OVERWRITE, z.ACC_NO_STORE | z.ACC_EMIT_BF16])
@pytest.mark.parametrize("vocab,cols,n,kind", [
    (50257, 300, 3000, "skewed"), (25001, 260, 17000, "skewed"), (30003, 125, 1000, "holes")])
def test_emb_grad_large_tables(vocab, cols, n, kind, flags, gaps):
    """Several rows of the table a wave, and one."""
    L, pl = layout(vocab * cols, gaps)
    ids = some_ids(kind, n, vocab, n)
    dy = torch.from_numpy(np.random.default_rng(n).integers(-4, 5, (n, cols))).to(BF16).to(DEV)
    f = Flat(L, pl, vocab * cols, DEV, ints=True)
    z.zero_embedding_grad(L, 1, torch.from_numpy(ids).to(DEV), dy, f.acc, 0.5, flags, f.out)
    g, _ = emb_exact(ids, f64(dy), vocab)
    f.check(g, np.zeros(g.size), 0.5, flags, f"{kind} {flags}")


@pytest.mark.parametrize("flags", [0, z.ACC_OVERWRITE])
@pytest.mark.parametrize("n", [1500, 16385, 40000])
def test_emb_grad_order_of_many_tokens(n, flags):
    test_emb_grad_is_the_same_every_time_and_in_token_order(n, flags)


@pytest.mark.parametrize("flags", [0, z.ACC_OVERWRITE])
@pytest.mark.parametrize("n", [1, 17, 300, 512, 513, 1024, 1025, 5000])
def test_emb_grad_is_the_same_every_time_and_in_token_order(n, flags):
    """Magnitudes from 2^-12 to 2^12: another order would give other bits.
    The stated order: pieces of 16 tokens, each ascending."""
    vocab, cols = 9, 260 if n % 2 else 1060
    L, pl = layout(vocab * cols, False)
    ids = some_ids("skewed", n, vocab, 4)
    dy = randn(6, n, cols, dtype=F32) * torch.exp2(torch.randint(-12, 13, (n, 1), device=DEV).float())
    got = []
    for _ in range(3):
        acc = torch.zeros(L.padded, device=DEV)
        z.zero_embedding_grad(L, 1, torch.from_numpy(ids).to(DEV), dy, acc, 1.0, flags)
        got.append(acc.cpu().numpy()[positions(pl, vocab * cols)].reshape(vocab, cols))
    assert np.array_equal(got[0], got[1]) and np.array_equal(got[0], got[2])
    d = dy.cpu().numpy()
    for v in range(vocab):
        rows = d[ids == v]
        total = np.zeros(cols, np.float32)
        pieces = []
        for k in range(0, len(rows), 16):
            s = np.zeros(cols, np.float32)
            for r in rows[k:k + 16]:
                s = s + r
            pieces.append(s)
        if len(pieces) == 1:
            total = pieces[0]
        else:
            for s in pieces:
                total = total + s
        assert np.array_equal(got[0][v], total), v


def test_emb_grad_rows_beyond_32_bits_and_no_tokens():
    vocab, cols = 300_001, 16_384
    L = z.Layout([vocab * cols], 0, 8, 0)
    acc = torch.zeros(L.padded, device=DEV)
    dy = randn(8, 3, cols)
    ids = torch.tensor([vocab - 1, vocab, vocab - 1], device=DEV)
    z.zero_embedding_grad(L, 0, ids, dy, acc, 1.0)
    assert torch.equal(acc[(vocab - 1) * cols:vocab * cols], dy[0].float() + dy[2].float())
    assert not acc[:1 << 20].any() and not acc[(vocab - 2) * cols:(vocab - 1) * cols].any()
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    z.zero_embedding_grad(L, 0, none, dy[:0], acc, 1.0, z.ACC_OVERWRITE)
    assert not acc.any()


def test_large_table_with_padding_inside_it():
    """4.9e9 elements in buckets of 12,500,003 (5 elements of padding each):
    rows on both sides of bucket borders and at the end of the table."""
    vocab, cols, cap, n_d = 300_001, 16_384, 12_500_003, 8
    L = z.Layout([vocab * cols], cap, n_d, 0)
    gap = -cap % n_d
    rows = sorted({0, 1, vocab - 1, vocab - 2} | {k * cap // cols + j for k in (1, 2, 77, 390)
                                                  for j in (-1, 0, 1)})
    x = torch.tensor(rows, device=DEV)[:, None] * cols + torch.arange(cols, device=DEV)
    at = x + x // cap * gap
    assert any(int(r[-1] - r[0]) != cols - 1 for r in at)      # a row that padding cuts
    params = torch.zeros(L.padded, dtype=BF16, device=DEV)
    vals = randn(5, len(rows), cols)
    params[at.reshape(-1)] = vals.reshape(-1)
    ids = torch.tensor(rows, device=DEV)
    out = torch.empty(len(rows), cols, dtype=BF16, device=DEV)
    z.zero_embedding_lookup(L, 0, params, ids, out)
    assert torch.equal(out, vals)
    del params
    acc = torch.zeros(L.padded, device=DEV)
    z.zero_embedding_grad(L, 0, ids, vals, acc)
    assert torch.equal(acc[at.reshape(-1)].view(-1, cols), vals.float())
    acc[at.reshape(-1)] = 0
    assert not acc.any()


# ------------------------------------------------------------------ norm
def norm_exact(x, res, w, eps):
    h = x if res is None else (x.float() + res.float()).to(BF16)
    hd = f64(h)
    with np.errstate(divide="ignore", invalid="ignore"):
        r = 1 / np.sqrt((hd ** 2).mean(1) + eps)
    return h, hd, r


NORM_SHAPES = [(1, 1), (3, 8), (5, 37), (2, 128), (9, 511), (9, 512), (6, 513), (333, 768),
               (4, 1024), (3, 1025), (5, 2048), (5, 2049), (3, 4096), (2, 4100), (3, 8192),
               (2, 8200), (2, 16384), (2, 16392), (2, 32768), (1100, 64)]


@pytest.mark.parametrize("gaps", [False, True])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_norm(gaps, rows, cols):
    L, pl = layout(cols, gaps and cols > 8)
    pos = torch.from_numpy(positions(pl, cols)).to(DEV)
    params = 1 + randn(cols, L.padded, scale=0.2)
    x, res = strided(randn(rows, rows, cols), 3, 1), strided(randn(rows + 1, rows, cols, scale=4.0), 0)
    res[:, ::50] *= 16
    eps = 1e-5
    for has_res in (True, False):
        h = torch.empty(rows, cols, dtype=BF16, device=DEV)
        y = torch.empty_like(h)
        rstd = torch.empty(rows, device=DEV)
        q, e = codes_like(rows, cols)
        z.zero_rms_norm(L, 1, params, x, res if has_res else None, eps, h, rstd, q, e, y)
        eh, hd, r = norm_exact(x, res if has_res else None, params, eps)
        assert torch.equal(h, eh)
        # a thread adds at most 32 squares, then 6 + 16 sums; the root halves that
        assert (np.abs(f64(rstd) - r) <= 40 * U * r).all()
        v = hd * r[:, None] * f64(params[pos])
        codes, scales = q.cpu().numpy(), e.cpu().numpy()
        got = act8_values(codes, scales)
        assert np.array_equal(f64(y), got)
        # the byte is that of the largest magnitude, but where this is within
        # the value's own error (44 U) of the border between two bytes
        lo, hi = act8(v * (1 - 44 * U))[1], act8(v * (1 + 44 * U))[1]
        assert ((scales == lo) | (scales == hi)).all()
        s = np.repeat(np.exp2(scales.astype(float) - 127), 128, axis=1)[:, :cols]
        lim = np.maximum(np.abs(v) * 2.0 ** -4, s * 2.0 ** -10) * (1 + 64 * U) + 44 * U * np.abs(v)
        assert (np.abs(got - v) <= lim).all()
        # without the optional outputs the codes are the same
        q2, e2 = codes_like(rows, cols)
        z.zero_rms_norm(L, 1, params, x, res if has_res else None, eps,
                        h if has_res else None, rstd, q2, e2)
        assert torch.equal(q, q2) and torch.equal(e, e2)


@pytest.mark.parametrize("rows,cols", [(200, 768), (64, 4096), (300, 129), (16, 16384)])
def test_norm_codes_are_the_rounded_exact_values(rows, cols):
    """Products and statistics are binary64, so a code differs from that of the
    64-bit reference only where the value is within about 2^-40 of itself of a
    halfway point: not among these inputs."""
    L, pl = layout(cols, False)
    pos = torch.from_numpy(positions(pl, cols)).to(DEV)
    params = 1 + randn(cols, L.padded, scale=0.2)
    x, res = randn(rows, rows, cols), randn(rows + 1, rows, cols, scale=4.0)
    h = torch.empty(rows, cols, dtype=BF16, device=DEV)
    rstd = torch.empty(rows, device=DEV)
    q, e = codes_like(rows, cols)
    z.zero_rms_norm(L, 1, params, x, res, 1e-5, h, rstd, q, e)
    _, hd, r = norm_exact(x, res, params, 1e-5)
    eq, ee = act8(hd * r[:, None] * f64(params[pos]))
    assert np.array_equal(e.cpu().numpy(), ee) and np.array_equal(q.cpu().numpy(), eq)
    assert np.array_equal(rstd.cpu().numpy(), r.astype(np.float32))


@pytest.mark.parametrize("size", [2.0 ** 100, 2.0 ** -60])
def test_norm_of_very_large_and_small_rows(size):
    """Squares and products with the weight that binary32 cannot hold."""
    rows, cols = 5, 400
    L, pl = layout(cols, False)
    pos = torch.from_numpy(positions(pl, cols)).to(DEV)
    params = (1 + randn(cols, L.padded, scale=0.2)) * size
    x = randn(rows, rows, cols) * size
    rstd = torch.empty(rows, device=DEV)
    q, e = codes_like(rows, cols)
    z.zero_rms_norm(L, 1, params, x, None, 0.0, None, rstd, q, e)
    _, hd, r = norm_exact(x, None, params, 0.0)
    eq, ee = act8(hd * r[:, None] * f64(params[pos]))
    assert np.array_equal(e.cpu().numpy(), ee) and np.array_equal(q.cpu().numpy(), eq)
    assert (np.abs(f64(rstd) - r) <= U * r).all()
    dy = randn(7, rows, cols)
    dx = torch.empty(rows, cols, dtype=BF16, device=DEV)
    f = Flat(L, pl, cols, DEV)
    z.zero_rms_norm_grad(L, 1, params, dy, None, x, rstd, dx, f.acc, 1.0)
    ex, lim, terms = norm_grad_exact(f64(dy), None, f64(x), f64(rstd)[:, None], f64(params[pos]))
    assert (np.abs(f64(dx) - ex) <= lim).all()
    f.check(terms.sum(0), (rows + 2) * U * np.abs(terms).sum(0), 1.0, 0, "weight")


def test_norm_zero_row_and_non_finite_row_stay_apart():
    rows, cols = 4, 300
    L, pl = layout(cols, False)
    params = torch.ones(L.padded, dtype=BF16, device=DEV)
    x = randn(1, rows, cols)
    x[1] = 0
    x[2, 7] = float("inf")
    rstd = torch.empty(rows, device=DEV)
    q, e = codes_like(rows, cols)
    y = torch.empty(rows, cols, dtype=BF16, device=DEV)
    z.zero_rms_norm(L, 1, params, x, None, 1e-5, None, rstd, q, e, y)
    r = 1 / np.sqrt(1e-5)
    assert not y[1].any() and abs(float(rstd[1]) - r) <= 4 * U * r + 2 * U * r  # eps in binary32
    assert float(rstd[2]) == 0 and torch.isnan(y[2, 7]) and not y[2, :7].any()
    q1, e1 = codes_like(1, cols)
    r1 = torch.empty(1, device=DEV)
    z.zero_rms_norm(L, 1, params, x[3:], None, 1e-5, None, r1, q1, e1)
    assert torch.equal(q[3:], q1) and torch.equal(e[3:], e1)


def norm_grad_exact(dy, dh, h, r, w):
    g = dy * w
    c = (g * h).mean(1, keepdims=True) * r * r
    dx = (0 if dh is None else dh) + r * (g - c * h)
    cols = h.shape[1]
    # binary32 before the rounding to bf16: the mean's sum has at most 32
    # terms a thread and 22 sums of threads, each term 2 products
    n = 64
    off_c = n * U * np.abs(g * h).mean(1, keepdims=True) * r * r
    off = r * (6 * U * (np.abs(g) + np.abs(c * h)) + off_c * np.abs(h)) + 2 * U * (
        0 if dh is None else np.abs(dh))
    return dx, BF * np.abs(dx) + (1 + BF) * (off + 3 * U * np.abs(dx)), dy * h * r


@pytest.mark.parametrize("gaps", [False, True])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES + [(5000, 100)])
def test_norm_grad(gaps, rows, cols):
    L, pl = layout(cols, gaps and cols > 8)
    pos = torch.from_numpy(positions(pl, cols)).to(DEV)
    params = 1 + randn(cols, L.padded, scale=0.2)
    h = randn(rows, rows, cols, scale=2.0)
    dy, dh = strided(randn(rows + 1, rows, cols), 1, 1), strided(randn(rows + 2, rows, cols), 2)
    r = torch.from_numpy(1 / np.sqrt((f64(h) ** 2).mean(1) + 1e-5)).float().to(DEV)
    for has_dh, flags in ((True, 0), (False, z.ACC_OVERWRITE | z.ACC_EMIT_BF16)):
        dx = torch.full((rows, cols), 5.0, dtype=BF16, device=DEV)
        f = Flat(L, pl, cols, DEV)
        z.zero_rms_norm_grad(L, 1, params, dy, dh if has_dh else None, h, r, dx, f.acc, 0.5, flags,
                             f.out)
        e, lim, terms = norm_grad_exact(f64(dy), f64(dh) if has_dh else None, f64(h),
                                        f64(r)[:, None], f64(params[pos]))
        assert (np.abs(f64(dx) - e) <= lim).all()
        f.check(terms.sum(0), (rows + 2) * U * np.abs(terms).sum(0), 0.5, flags, "weight")


# several rows a block and several turns of it, the last ones short, at widths
# on both sides of each change of the rows' threads
NORM_MANY = [(533, 128), (17, 129), (16500, 130), (531, 256), (4100, 257), (77, 1000), (4105, 640),
             (33, 2000), (2051, 1300), (1027, 2300), (1026, 4096), (515, 4104), (2060, 5000),
             (5, 6144), (5, 6152), (514, 8200), (9, 12288), (9, 12296), (261, 16400), (9, 24576),
             (1030, 24584)]


@pytest.mark.parametrize("rows,cols", NORM_MANY)
def test_norm_of_many_rows(rows, cols):
    test_norm(rows % 2 == 1, rows, cols)


@pytest.mark.parametrize("rows,cols", NORM_MANY)
def test_norm_grad_of_many_rows(rows, cols):
    test_norm_grad(rows % 2 == 1, rows, cols)
    test_norm_grad(rows % 2 == 0, min(rows, 40), cols)


@pytest.mark.parametrize("flags", FLAG_SETS)
def test_norm_grad_flags_and_no_rows(flags):
    rows, cols = 40, 70
    L, pl = layout(cols, True)
    params = randn(1, L.padded)
    h, dy = randn(2, rows, cols), randn(3, rows, cols)
    r = torch.ones(rows, device=DEV)
    for n in (rows, 0):
        f = Flat(L, pl, cols, DEV)
        dx = torch.empty(n, cols, dtype=BF16, device=DEV)
        z.zero_rms_norm_grad(L, 1, params, dy[:n], None, h[:n], r[:n], dx, f.acc, 2.0, flags, f.out)
        t = f64(dy[:n]) * f64(h[:n])
        f.check(t.sum(0), (n + 2) * U * np.abs(t).sum(0), 2.0, flags, f"rows {n}")


def test_norm_grad_against_differences():
    """Central differences of the unrounded norm, in 64 bits."""
    rows, cols = 6, 200
    L, pl = layout(cols, False)
    params = 1 + randn(1, L.padded, scale=0.2)
    w = f64(params)[positions(pl, cols)]
    h, dy = randn(2, rows, cols), randn(3, rows, cols)
    hd, gd = f64(h), f64(dy)
    eps = 1e-5

    def loss(hh, ww):
        return (gd * hh / np.sqrt((hh ** 2).mean(1, keepdims=True) + eps) * ww).sum()

    r = torch.from_numpy(1 / np.sqrt((hd ** 2).mean(1) + eps)).float().to(DEV)
    dx = torch.empty_like(h)
    acc = torch.zeros(L.padded, device=DEV)
    z.zero_rms_norm_grad(L, 1, params, dy, None, h, r, dx, acc, 1.0)
    gx, gw = f64(dx), f64(acc)[positions(pl, cols)]
    rng = np.random.default_rng(5)
    t = 1e-4
    for _ in range(5):
        a, b = rng.standard_normal(hd.shape), rng.standard_normal(cols)
        dl = (loss(hd + t * a, w) - loss(hd - t * a, w)) / (2 * t)
        # rounding of dx to bf16, and the differences' own error (t^2)
        assert abs((gx * a).sum() - dl) <= BF * np.abs(gx * a).sum() + 1e-5 * np.abs(gx * a).sum()
        dl = (loss(hd, w + t * b) - loss(hd, w - t * b)) / (2 * t)
        assert abs((gw * b).sum() - dl) <= 1e-5 * np.abs(gw * b).sum()


# ------------------------------------------------------------------ weight gradient
LINEAR_SHAPES = [(1, 1, 1), (2, 3, 5), (64, 32, 32), (63, 33, 31), (65, 128, 128), (100, 129, 127),
                 (16, 300, 7), (16, 7, 300), (257, 256, 512), (700, 130, 260), (2048, 64, 48),
                 (3000, 257, 129), (1, 1000, 1000), (130, 513, 640),
                 (200, 1, 1), (129, 1, 3), (256, 5, 16), (193, 8, 1), (640, 519, 271)]


@pytest.mark.parametrize("tr", [False, True])
@pytest.mark.parametrize("gaps", [False, True])
@pytest.mark.parametrize("tokens,o,i", LINEAR_SHAPES)
def test_linear_grad_exact_in_integers(tr, gaps, tokens, o, i):
    """dY in -3..3, X in -8..8 times a power of two per block: every sum is a
    small multiple of one, exact in any order."""
    r = np.random.default_rng(tokens + o)
    L, pl = layout(o * i, gaps and o * i > 8)
    dy = strided(torch.from_numpy(r.integers(-3, 4, (tokens, o))).to(BF16).to(DEV), 3, 1)
    xi = r.integers(-8, 9, (tokens, i))
    xi[:, ::128] = 448                     # every block has the scale 1
    q, e = codes_like(tokens, i)
    z.zero_act8_pack(torch.from_numpy(xi).to(F32).to(DEV), q, e)
    shift = r.integers(0, 3, e.shape)
    e += torch.from_numpy(shift).to(DEV).to(U8)
    xv = act8_values(q.cpu().numpy(), e.cpu().numpy())
    assert np.array_equal(xv, np.round(xv))
    g = f64(dy).T @ xv
    assert np.abs(f64(dy)).T.max(initial=0) * np.abs(xv).sum(0).max() < 2 ** 24
    g = (g.T if tr else g).reshape(-1)
    for flags in (0, z.ACC_OVERWRITE):
        f = Flat(L, pl, o * i, DEV, ints=True)
        z.zero_linear_grad(L, 1, dy, q, e, f.acc, 1.0, flags, f.out, transposed=tr)
        f.check(g, 0.0, 1.0, flags, f"{tokens} {o} {i}")
        exp = g if flags else f.acc0[f.pos] + g
        assert np.array_equal(f64(f.acc)[f.pos], exp)


@pytest.mark.parametrize("flags", FLAG_SETS)
@pytest.mark.parametrize("tokens,o,i,gaps", [(300, 70, 90, True), (300, 128, 256, False),
                                             (0, 33, 65, True), (0, 33, 64, False),
                                             (2500, 40, 40, False)])
def test_linear_grad_flags(flags, tokens, o, i, gaps):
    L, pl = layout(o * i, gaps)
    dy, x = randn(1, tokens, o), randn(2, tokens, i, scale=3.0)
    q, e = codes_like(tokens, i)
    z.zero_act8_pack(x, q, e)
    xv = act8_values(q.cpu().numpy(), e.cpu().numpy())
    f = Flat(L, pl, o * i, DEV)
    z.zero_linear_grad(L, 1, dy, q.view(F8), e, f.acc, 0.25, flags, f.out)
    d = f64(dy)
    # twice the rounded sum's bound: the matrix cores' own sums need not round to nearest
    f.check((d.T @ xv).reshape(-1), (2 * (tokens + 8) * U * (np.abs(d).T @ np.abs(xv))).reshape(-1),
            0.25, flags, "linear")


@pytest.mark.parametrize("tr", [False, True])
def test_linear_grad_large_tiles_and_dim0_layout(tr):
    """Sizes of several tiles with odd edges, in a per-parameter layout."""
    tokens, o, i = 1500, 1100, 900
    L, pl = layout(o * i, False, dim0_rows=i if tr else o)
    r = np.random.default_rng(0)
    dy = torch.from_numpy(r.integers(-3, 4, (tokens, o))).to(BF16).to(DEV)
    xi = r.integers(-8, 9, (tokens, i))
    q, e = codes_like(tokens, i)
    z.zero_act8_pack(torch.from_numpy(xi).to(BF16).to(DEV), q, e)
    xv = act8_values(q.cpu().numpy(), e.cpu().numpy())
    assert np.array_equal(xv, xi)
    g = f64(dy).T @ xv
    f = Flat(L, pl, o * i, DEV, ints=True)
    z.zero_linear_grad(L, 1, dy, q, e, f.acc, 1.0, transposed=tr)
    assert np.array_equal(f64(f.acc)[f.pos], f.acc0[f.pos] + (g.T if tr else g).reshape(-1))


@pytest.mark.parametrize("tr", [False, True])
@pytest.mark.parametrize("gaps", [False, True])
@pytest.mark.parametrize("tokens,o,i", [(1300, 4200, 4090), (1000, 4096, 4096), (700, 4100, 4090),
                                        (20_000, 520, 1030), (513, 5000, 3100)])
def test_linear_grad_sizes_of_both_tiles_exact_in_integers(tr, gaps, tokens, o, i):
    """Sizes that take the 256-column tile, the 128-column tile, whole tiles
    only, and whole and split ones, with every edge ragged or none."""
    g = torch.Generator(device=DEV).manual_seed(tokens)
    dy = torch.randint(-3, 4, (tokens, o), generator=g, device=DEV).to(BF16)
    x = torch.randint(-8, 9, (tokens, i), generator=g, device=DEV).float()
    q, e = codes_like(tokens, i)
    z.zero_act8_pack(x, q, e)
    L, pl = layout(o * i, gaps)
    pos = torch.from_numpy(positions(pl, o * i)).to(DEV)
    exact = dy.double().t().contiguous() @ x.double()          # below 2^53: exact
    assert float(exact.abs().max()) < 2 ** 24 and 24 * tokens < 2 ** 24
    exact = (exact.t() if tr else exact).reshape(-1)
    acc = torch.randint(-9, 10, (L.padded,), generator=g, device=DEV).float()
    out = torch.full((L.padded,), 3.0, dtype=BF16, device=DEV)
    start = acc.clone()
    z.zero_linear_grad(L, 1, dy, q, e, acc, 1.0, z.ACC_EMIT_BF16, out, transposed=tr)
    exp = start.double()
    exp[pos] += exact
    assert torch.equal(acc.double(), exp)
    rest = torch.ones(L.padded, dtype=torch.bool, device=DEV)
    rest[pos] = False
    assert torch.equal(out[pos], exp[pos].float().to(BF16)) and (out[rest] == 3.0).all()


def test_linear_grad_non_finite_inputs_reach_only_their_row_and_column():
    tokens, o, i = 200, 150, 170
    L, pl = layout(o * i, False)
    dy, x = randn(1, tokens, o), randn(2, tokens, i)
    x[50, 33] = float("nan")
    dy[77, 5] = float("inf")
    q, e = codes_like(tokens, i)
    z.zero_act8_pack(x, q, e)
    acc = torch.zeros(L.padded, device=DEV)
    z.zero_linear_grad(L, 1, dy, q, e, acc)
    bad = ~np.isfinite(f64(acc)[positions(pl, o * i)].reshape(o, i))
    exp = np.zeros_like(bad)
    exp[:, 33] = True
    exp[5, :] = True
    assert np.array_equal(bad, exp)


@pytest.mark.parametrize("a,b", [(2.0 ** -130, 2.0 ** 10), (2.0 ** -133, 2.0 ** 20),
                                 (2.0 ** -100, 2.0 ** -30), (-2.0 ** -127, 1.0),
                                 (2.0 ** -64, 2.0 ** -64)])
def test_linear_grad_keeps_subnormals(a, b):
    """bf16 inputs, products and sums below the normal range are exact too."""
    L = z.Layout([8 * 16], 0, 1, 0)
    dy, x = torch.zeros(20, 8, dtype=BF16, device=DEV), torch.zeros(20, 16, device=DEV)
    dy[3], x[3] = a, b
    q, e = codes_like(20, 16)
    z.zero_act8_pack(x, q, e)
    acc = torch.zeros(128, device=DEV)
    z.zero_linear_grad(L, 0, dy, q, e, acc)
    assert (acc.double() == a * b).all()


def test_linear_grad_inputs_beyond_32_bits():
    tokens, o, i = 70_000, 65_536, 32     # dY: 4.6e9 elements
    L = z.Layout([o * i], 0, 8, 0)
    dy = torch.zeros(tokens, o, dtype=BF16, device=DEV)
    q, e = torch.zeros(tokens, i, dtype=U8, device=DEV), torch.full((tokens, 1), 127, dtype=U8, device=DEV)
    q[-1] = 0x38                           # 1.0
    dy[-1] = torch.arange(o, device=DEV) % 251
    acc = torch.zeros(L.padded, device=DEV)
    z.zero_linear_grad(L, 0, dy, q, e, acc, 2.0)
    exp = (torch.arange(o, device=DEV) % 251).float() * 2
    assert torch.equal(acc[:o * i].view(o, i), exp[:, None].expand(o, i))


def test_linear_grad_against_differences():
    """The product is linear in the weight: L(W + d) - L(W) = <dW, d>."""
    tokens, o, i = 90, 40, 60
    L, pl = layout(o * i, False)
    dy, x = randn(1, tokens, o), randn(2, tokens, i)
    q, e = codes_like(tokens, i)
    z.zero_act8_pack(x, q, e)
    acc = torch.zeros(L.padded, device=DEV)
    z.zero_linear_grad(L, 1, dy, q, e, acc)
    g = f64(acc)[positions(pl, o * i)].reshape(o, i)
    xv, d = act8_values(q.cpu().numpy(), e.cpu().numpy()), f64(dy)
    w, a = np.random.default_rng(1).standard_normal((2, o, i))
    diff = (d * (xv @ (w + a).T)).sum() - (d * (xv @ w.T)).sum()
    mag = (np.abs(d).T @ np.abs(xv) * np.abs(a)).sum()
    assert abs((g * a).sum() - diff) <= 2 * (tokens + 8) * U * mag + 1e-9 * mag


# ------------------------------------------------------------------ together
class Net:
    """Table -> norm (with the residual) -> linear, two micro-batches, in one
    bucketed layout whose buckets cut the tensors: what a data-parallel rank
    does between its batches and its step."""
    VOCAB, D, O, T = 90, 72, 40, 50

    def __init__(self, seed=0):
        V, D, O = self.VOCAB, self.D, self.O
        self.numel = [V * D, D, O * D]
        self.cap, self.n_d = 2501, 2
        self.pl = oracle.plan(self.numel, self.cap, self.n_d)
        self.L = [z.Layout(self.numel, self.cap, self.n_d, r) for r in range(2)]
        self.params = randn(seed, self.L[0].padded, scale=0.3)
        off = np.concatenate([[0], np.cumsum(self.numel)])
        x = np.arange(off[-1])
        b = np.searchsorted(self.pl.stream_off, x, side="right") - 1
        flat = np.asarray(self.pl.padded_off)[b] + x - np.asarray(self.pl.stream_off)[b]
        self.pos = [flat[off[t]:off[t + 1]] for t in range(3)]

    def tensor(self, flat, t, *shape):
        return f64(flat)[self.pos[t]].reshape(shape)

    def batch(self, seed):
        g = torch.Generator().manual_seed(seed)
        ids = torch.randint(-1, self.VOCAB, (self.T,), generator=g)
        return ids.to(DEV), randn(seed + 1, self.T, self.D), randn(seed + 2, self.T, self.O, scale=0.1)

    def buffers(self):
        T, D, new = self.T, self.D, lambda *s, dtype=BF16: torch.empty(*s, dtype=dtype, device=DEV)
        return dict(x=new(T, D), h=new(T, D), y=new(T, D), dx=new(T, D), rstd=new(T, dtype=F32),
                    q=new(T, D, dtype=U8), e=new(T, 1, dtype=U8))

    def forward_backward(self, ids, res, dout, acc, b, scale, flags=0, out=None, stream=None):
        L, kw = self.L[0], {"stream": stream}
        z.zero_embedding_lookup(L, 0, self.params, ids, b["x"], 4.0, **kw)
        z.zero_rms_norm(L, 1, self.params, b["x"], res, 1e-5, b["h"], b["rstd"], b["q"], b["e"],
                        b["y"], **kw)
        W = self.W
        dy = dout @ W                                  # the linear layer's input gradient
        z.zero_linear_grad(L, 2, dout, b["q"], b["e"], acc, scale, flags, out, **kw)
        z.zero_rms_norm_grad(L, 1, self.params, dy, None, b["h"], b["rstd"], b["dx"], acc, scale,
                             flags, out, **kw)
        z.zero_embedding_grad(L, 0, ids, b["dx"], acc, 4.0 * scale, flags, out, **kw)
        return dy

    @property
    def W(self):
        if not hasattr(self, "_w"):
            self._w = self.params[torch.from_numpy(self.pos[2]).to(DEV)].view(self.O, self.D).contiguous()
        return self._w

    def exact(self, ids, res, dout, b, dy):
        """Gradients by the formulas in 64 bits, from the values each call read."""
        V, D, O = self.VOCAB, self.D, self.O
        xv = act8_values(b["q"].cpu().numpy(), b["e"].cpu().numpy())
        h, r, w = f64(b["h"]), f64(b["rstd"])[:, None], self.tensor(self.params, 1, D)
        table, _ = emb_exact(ids.cpu().numpy(), f64(b["dx"]), V)
        return [4.0 * table, (f64(dy) * h * r).sum(0), (f64(dout).T @ xv).reshape(-1)]


def test_two_micro_batches_then_the_step():
    """OVERWRITE, then add with emission in bf16: the emitted flat buffer is
    the rank's contribution, stepped by zero_shard_step against the oracle."""
    net = Net()
    P = net.L[0].padded
    contrib = []
    for rank in range(2):
        acc = torch.zeros(P, device=DEV)
        out = torch.zeros(P, dtype=BF16, device=DEV)
        total = [0.0] * 3
        for mb, flags in ((0, z.ACC_OVERWRITE), (1, z.ACC_EMIT_BF16 | z.ACC_NO_STORE)):
            b = net.buffers()
            ids, res, dout = net.batch(10 * rank + 100 * mb)
            dy = net.forward_backward(ids, res, dout, acc, b, 0.5, flags, out)
            tab = net.tensor(net.params, 0, net.VOCAB, net.D)
            idc = ids.cpu().numpy()
            lk = np.where((idc >= 0)[:, None], tab[np.maximum(idc, 0)] * 4.0, 0.0)
            assert np.array_equal(f64(b["x"]), lk)      # a power of two: exact
            total = [t + 0.5 * g for t, g in zip(total, net.exact(ids, res, dout, b, dy))]
        for t in range(3):
            got = f64(out)[net.pos[t]]
            # two sums of up to 100 products of magnitude up to some units: far
            # below bf16's half step, but near zero
            assert np.abs(got - total[t]).max() <= BF * np.abs(total[t]).max()
            big = np.abs(total[t]) > 1e-3 * np.abs(total[t]).max()
            assert (np.abs(got - total[t])[big] <= 1.01 * BF * np.abs(total[t])[big]).all()
        contrib.append(out)
    flat = [c.view(torch.int16).cpu().numpy().view(np.uint16) for c in contrib]
    hp = z.AdamW()
    for rank in range(2):
        L = net.L[rank]
        S = L.shard
        th, m, v = (torch.zeros(S, device=DEV) for _ in range(3))
        th.normal_()
        p = torch.zeros(P, dtype=torch.int16, device=DEV)
        fp, _ = net.pl.map(rank, np.arange(S))
        oth, om, ov = (t.cpu().numpy().copy() for t in (th, m, v))
        z.zero_shard_step(L, hp, 1, contrib, z.GRAD_FLAT, th, m, v, p, z.OUT_AG_SLOT)
        op, _ = oracle.shard_step([np.ascontiguousarray(f[fp]) for f in flat], oth, om, ov,
                                  oracle.AdamW(), 1, want_grad=True)
        assert np.array_equal(th.cpu().numpy(), oth)
        assert np.array_equal(p.cpu().numpy().view(np.uint16)[fp], op)


@pytest.mark.parametrize("tokens", [50, 700])
def test_captured_and_replayed_with_eager_work_between(tokens):
    net = Net(3)
    net.T = tokens
    P = net.L[0].padded
    batches = [net.batch(s) for s in (1, 2, 3, 4)]
    ids, res, dout = (t.clone() for t in batches[0])
    b, acc = net.buffers(), torch.zeros(P, device=DEV)
    side = torch.cuda.Stream()
    net.W
    ws = [torch.empty(1 << 20, dtype=U8, device=DEV) for _ in range(3)]
    L = net.L[0]

    def body(stream=None):
        z.zero_embedding_lookup(L, 0, net.params, ids, b["x"], 4.0, stream=stream)
        z.zero_rms_norm(L, 1, net.params, b["x"], res, 1e-5, b["h"], b["rstd"], b["q"], b["e"],
                        b["y"], stream=stream)
        z.zero_linear_grad(L, 2, dout, b["q"], b["e"], acc, 0.5, workspace=ws[0], stream=stream)
        z.zero_rms_norm_grad(L, 1, net.params, b["y"], None, b["h"], b["rstd"], b["dx"], acc, 0.5,
                             workspace=ws[1], stream=stream)
        # without a workspace: allocated in the graph's own memory
        z.zero_embedding_grad(L, 0, ids, b["dx"], acc, 0.5, stream=stream)

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        body()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        body()
    for bt in batches + batches[:2]:
        for to, src in zip((ids, res, dout), bt):
            to.copy_(src)
        acc.normal_()
        start = acc.clone()
        graph.replay()
        torch.cuda.synchronize()
        got = acc.clone()
        dx = b["dx"].clone()
        acc.copy_(start)
        body()
        torch.cuda.synchronize()
        assert torch.equal(acc, got) and torch.equal(b["dx"], dx)
        torch.randn(1000, device=DEV).sum().item()     # the program's own work between


@pytest.mark.parametrize("flags", [0, z.ACC_OVERWRITE])
def test_many_tokens_captured_and_replayed(flags):
    vocab, cols, n = 2000, 130, 20000
    L, _ = layout(vocab * cols, True)
    ids = torch.from_numpy(some_ids("skewed", n, vocab, 1)).to(DEV)
    dy, acc = randn(1, n, cols), torch.zeros(L.padded, device=DEV)

    def body():
        z.zero_embedding_grad(L, 1, ids, dy, acc, 0.5, flags)

    body()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    for k, kind in enumerate(("uniform", "skewed", "same", "holes", "uniform")):
        ids.copy_(torch.from_numpy(some_ids(kind, n, vocab, k)).to(DEV))
        dy.copy_(randn(k + 5, n, cols))
        acc.normal_()
        start = acc.clone()
        graph.replay()
        torch.cuda.synchronize()
        got = acc.clone()
        acc.copy_(start)
        body()
        torch.cuda.synchronize()
        assert torch.equal(acc, got)
        torch.randn(1000, device=DEV).sum().item()


@pytest.mark.parametrize("tokens", [50, 700])
def test_other_streams(tokens):
    """A call on a stream that is not the current one, with its own
    workspace allocation, gives the same bits."""
    net = Net(5)
    net.T = tokens
    ids, res, dout = net.batch(9)
    acc = [torch.zeros(net.L[0].padded, device=DEV) for _ in range(2)]
    net.W
    net.forward_backward(ids, res, dout, acc[0], net.buffers(), 0.5)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = net.buffers()
        dy = dout @ net.W
        side.synchronize()
    net_W = net._w
    L = net.L[0]
    z.zero_embedding_lookup(L, 0, net.params, ids, b["x"], 4.0, stream=side)
    z.zero_rms_norm(L, 1, net.params, b["x"], res, 1e-5, b["h"], b["rstd"], b["q"], b["e"], b["y"],
                    stream=side)
    z.zero_linear_grad(L, 2, dout, b["q"], b["e"], acc[1], 0.5, stream=side)
    z.zero_rms_norm_grad(L, 1, net.params, dy, None, b["h"], b["rstd"], b["dx"], acc[1], 0.5,
                         stream=side)
    z.zero_embedding_grad(L, 0, ids, b["dx"], acc[1], 2.0, stream=side)
    torch.cuda.synchronize()
    assert net_W is net.W and torch.equal(acc[0], acc[1])
