"""The micro-batch operators on the GPU at the edges of their kernels: last,
partly filled groups of columns, turns of a block, addresses, calls at the same
time."""
import threading

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_step_amd as z
from micrograd_ref import Flat, U, act8, act8_values, f64, layout
from test_gpu_micrograd import BF16, DEV, emb_exact, some_ids

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free_gpu_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def small_ints(seed, *shape, dtype=BF16):
    return torch.from_numpy(np.random.default_rng(seed).integers(-4, 5, shape)).to(dtype).to(DEV)


@pytest.mark.parametrize("gaps", [False, True])
@pytest.mark.parametrize("flags", [0, z.ACC_OVERWRITE, z.ACC_EMIT_BF16])
@pytest.mark.parametrize("cols", [125, 128, 253, 256, 257, 260, 261, 509, 513, 772])
def test_emb_grad_of_rows_that_leave_lanes_without_columns(cols, flags, gaps):
    """A wave takes 256 columns; the last one of a row as few as one.  Ids of
    one token, of several pieces and of 1024 tokens and more; sums of small
    integers, exact in any order."""
    vocab, n = 90, 2600
    ids = some_ids("uniform", n, vocab, cols)
    ids[100:1300] = 7
    ids[1300:1320] = 8
    ids[::13] = -1
    L, pl = layout(vocab * cols, gaps)
    dy = small_ints(cols, n, cols)
    f = Flat(L, pl, vocab * cols, DEV, ints=True)
    z.zero_embedding_grad(L, 1, torch.from_numpy(ids).to(DEV), dy, f.acc, 1.0, flags, f.out)
    g, _ = emb_exact(ids, f64(dy), vocab)
    want = (0 if flags & z.ACC_OVERWRITE else f.acc0[f.pos]) + g
    assert np.array_equal(f64(f.acc)[f.pos], want)
    f.check(g, np.zeros(g.size), 1.0, flags, f"{cols}")


# ------------------------------------------------------------------ addresses
class At:
    """A tensor's bytes `shift` bytes into a buffer of their own."""

    def __init__(self, t, shift):
        t = t.contiguous()
        self.dtype, self.shape, self.shift = t.dtype, t.shape, shift
        self.n = t.numel() * t.element_size()
        self.buf = torch.full((self.n + 64,), 0xA5, dtype=torch.uint8, device=DEV)
        self.buf[shift:shift + self.n] = t.to(DEV).view(-1).view(torch.uint8)

    @property
    def p(self):
        return self.buf.data_ptr() + self.shift

    def get(self):
        assert (self.buf[:self.shift] == 0xA5).all() and (self.buf[self.shift + self.n:] == 0xA5).all()
        return self.buf[self.shift:self.shift + self.n].clone().view(self.dtype).view(self.shape)


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("shift", [1, 2, 4, 7])
@pytest.mark.parametrize("id_dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("n,cols,flags", [(1, 8, 0), (60, 37, 0), (512, 260, 0), (600, 260, 0),
                                          (700, 37, z.ACC_OVERWRITE | z.ACC_EMIT_BF16)])
def test_embedding_at_any_address(n, cols, flags, id_dtype, shift):
    """Through the C entry points: torch's own tensors are aligned."""
    vocab = 300
    lib, L = z.load(), z.Layout([vocab * cols], 0, 4, 0)
    ids = torch.from_numpy(some_ids("skewed", n, vocab, 3)).to(id_dtype)
    ids[n // 2] = vocab - 1
    table, dy = small_ints(1, L.padded), small_ints(2, n, cols)
    acc, out = small_ints(3, L.padded, dtype=torch.float32), torch.zeros(L.padded, dtype=BF16)
    i, t, d, a, o = (At(x, shift) for x in (ids, table, dy, acc, out))
    x = At(torch.zeros(n, cols, dtype=BF16), shift)
    size = ids.element_size()
    assert lib.zero_embedding_lookup(L.handle, 0, cols, t.p, i.p, size, n, 1.0, x.p, cols, 0, stream()) == 0
    ws = torch.empty(lib.zero_embedding_grad_workspace(L.handle, 0, cols, n, flags) + 16,
                     dtype=torch.uint8, device=DEV)
    assert lib.zero_embedding_grad(L.handle, 0, cols, i.p, size, n, d.p, cols, 0, 1.0, flags, a.p, o.p,
                                   ws.data_ptr(), ws.numel(), stream()) == 0
    rows = table[:vocab * cols].view(vocab, cols)
    assert torch.equal(x.get(), rows[ids.long().to(DEV)])
    g, _ = emb_exact(ids.numpy(), f64(dy), vocab)
    want = (0 if flags & z.ACC_OVERWRITE else f64(acc)[:vocab * cols]) + g
    assert np.array_equal(f64(a.get())[:vocab * cols], want)
    if flags & z.ACC_EMIT_BF16:
        assert torch.equal(o.get()[:vocab * cols], a.get()[:vocab * cols].to(BF16))
    else:
        assert not o.get().any()


@pytest.mark.parametrize("shift", [1, 2, 7])
@pytest.mark.parametrize("rows,cols", [(1, 8), (5, 37), (9, 768), (40, 2056)])
def test_norm_and_act8_at_any_address(rows, cols, shift):
    """The same bits as from aligned memory."""
    lib, L = z.load(), z.Layout([cols], 0, 4, 0)
    r = np.random.default_rng(rows)
    real = lambda *s, dtype=BF16: torch.from_numpy(r.standard_normal(s)).to(dtype).to(DEV)  # noqa: E731
    w, x, res, dy, dh = real(L.padded), *(real(rows, cols) for _ in range(4))
    a0, nb = real(L.padded, dtype=torch.float32), -(-cols // 128)
    got = []
    for s in (0, shift):
        W, X, R, DY, DH, ACC = (At(t, s) for t in (w, x, res, dy, dh, a0))
        H, Y, DX, V = (At(torch.zeros(rows, cols, dtype=BF16), s) for _ in range(4))
        Q, E = At(torch.zeros(rows, cols, dtype=torch.uint8), s), At(torch.zeros(rows, nb, dtype=torch.uint8), s)
        RS, XF, VF = (At(t, s) for t in (torch.zeros(rows), x.float(), torch.zeros(rows, cols)))
        Q2, E2 = At(torch.zeros(rows, cols, dtype=torch.uint8), s), At(torch.zeros(rows, nb, dtype=torch.uint8), s)
        h = L.handle
        assert lib.zero_rms_norm(h, 0, W.p, X.p, cols, R.p, cols, rows, 1e-5, H.p, RS.p, Q.p, E.p,
                                 Y.p, stream()) == 0
        ws = torch.empty(lib.zero_rms_norm_grad_workspace(h, 0, rows) + 16, dtype=torch.uint8, device=DEV)
        assert lib.zero_rms_norm_grad(h, 0, W.p, DY.p, cols, DH.p, cols, H.p, RS.p, rows, 0.5, 0, DX.p,
                                      ACC.p, None, ws.data_ptr(), ws.numel(), stream()) == 0
        assert lib.zero_act8_unpack(Q.p, E.p, rows, cols, V.p, 0, cols, stream()) == 0
        assert lib.zero_act8_pack(XF.p, 1, rows, cols, cols, Q2.p, E2.p, stream()) == 0
        assert lib.zero_act8_unpack(Q2.p, E2.p, rows, cols, VF.p, 1, cols, stream()) == 0
        assert torch.equal(Y.get(), V.get())
        got.append([t.get() for t in (H, Y, DX, Q, E, RS, ACC, Q2, E2, VF)])
    for a, b in zip(*got):
        assert torch.equal(a, b) and a.float().abs().sum() > 0


@pytest.mark.parametrize("tr", [0, 1])
@pytest.mark.parametrize("shift", [1, 2, 7])
@pytest.mark.parametrize("tokens,o,i", [(1, 3, 5), (70, 33, 130), (300, 256, 512), (1000, 300, 260),
                                        (700, 4100, 4090)])
def test_linear_grad_at_any_address(tokens, o, i, shift, tr):
    lib, L = z.load(), z.Layout([o * i], 0, 4, 0)
    dy, x = small_ints(tokens, tokens, o), small_ints(i, tokens, i)
    a0 = small_ints(o, L.padded, dtype=torch.float32)
    q = torch.empty(tokens, i, dtype=torch.uint8, device=DEV)
    e = torch.empty(tokens, -(-i // 128), dtype=torch.uint8, device=DEV)
    z.zero_act8_pack(x, q, e)
    D, Q, E, A, O = (At(t, shift) for t in (dy, q, e, a0, torch.zeros(L.padded, dtype=BF16)))
    ws = torch.empty(lib.zero_linear_grad_workspace(L.handle, 0, tr, o, i, tokens) + 16,
                     dtype=torch.uint8, device=DEV)
    assert lib.zero_linear_grad(L.handle, 0, tr, D.p, o, Q.p, E.p, tokens, o, i, 1.0, z.ACC_EMIT_BF16,
                                A.p, O.p, ws.data_ptr(), ws.numel(), stream()) == 0
    g = dy.double().t().contiguous() @ x.double()              # sums below 16 * 1000: exact
    want = a0.double()
    want[:o * i] += (g.t() if tr else g).reshape(-1)
    assert torch.equal(A.get().double(), want)
    assert torch.equal(O.get()[:o * i], want[:o * i].float().to(BF16))


# ------------------------------------------------------------------ turns of a block
def codes_like(rows, cols):
    return (torch.full((rows, cols), 0x55, dtype=torch.uint8, device=DEV),
            torch.full((rows, -(-cols // 128)), 0x55, dtype=torch.uint8, device=DEV))


# a launch has at most 16384 blocks of 16, 8, 4 or 1 rows: two or three turns of
# a block, the last one short
@pytest.mark.parametrize("rows,cols,per_turn", [
    (262_150, 12, 16 << 14), (131_080, 200, 8 << 14), (65_541, 520, 4 << 14),
    (16_389, 1032, 1 << 14), (33_000, 1032, 1 << 14), (16_390, 4104, 1 << 14),
    (16_385, 8200, 1 << 14), (16_387, 16_392, 1 << 14)])
def test_norm_of_more_rows_than_a_launch_has_blocks_for(rows, cols, per_turn):
    """Every row as in a call on fewer rows, which one turn covers, and rows on
    both sides of a turn as the 64-bit reference has them, the codes exactly and
    1/rms by one rounding to binary32 (2^-24 of it, and what binary64 adds)."""
    g = torch.Generator(device=DEV).manual_seed(cols)
    real = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF16)  # noqa: E731
    L = z.Layout([cols], 0, 4, 0)
    params, x, res = 1 + 0.2 * real(L.padded), real(rows, cols), 4 * real(rows, cols)
    x *= torch.exp2(torch.randint(-6, 7, (rows, 1), generator=g, device=DEV).float()).to(BF16)

    def norm(a, b):
        h, y = (torch.empty(b - a, cols, dtype=BF16, device=DEV) for _ in range(2))
        rstd, (q, e) = torch.empty(b - a, device=DEV), codes_like(b - a, cols)
        z.zero_rms_norm(L, 0, params, x[a:b], res[a:b], 1e-5, h, rstd, q, e, y)
        return h, rstd, q, e, y

    whole = norm(0, rows)
    for a in range(0, rows, per_turn // 2):
        b = min(rows, a + per_turn // 2)
        for t, part in zip(whole, norm(a, b)):
            assert torch.equal(t[a:b], part), f"rows {a} to {b}"
    at = sorted({0, 1, rows - 1, rows - 2} | {k * per_turn + j for k in range(1, rows // per_turn + 1)
                                              for j in (-2, -1, 0, 1, 2) if k * per_turn + j < rows})
    at = torch.tensor(at, device=DEV)
    h = (x[at].float() + res[at].float()).to(BF16)
    hd = f64(h)
    r = 1 / np.sqrt((hd ** 2).mean(1) + 1e-5)
    eq, ee = act8(hd * r[:, None] * f64(params[:cols]))
    assert torch.equal(whole[0][at], h)
    assert (np.abs(f64(whole[1][at]) - r) <= U * r * (1 + 2.0 ** -20)).all()
    assert np.array_equal(whole[2][at].cpu().numpy(), eq)
    assert np.array_equal(whole[3][at].cpu().numpy(), ee)


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_act8_of_more_blocks_than_a_launch_takes_at_once(dtype):
    rows, cols = 40_001, 1033                        # 360009 blocks of 128, 262144 at once
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(rows, cols, generator=g, device=DEV).to(dtype)
    (q, e), out = codes_like(rows, cols), torch.empty(rows, cols, dtype=dtype, device=DEV)
    z.zero_act8_pack(x, q, e)
    z.zero_act8_unpack(q, e, out)
    for a in range(0, rows, 20_000):
        b = min(rows, a + 20_000)
        (q1, e1), o1 = codes_like(b - a, cols), torch.empty(b - a, cols, dtype=dtype, device=DEV)
        z.zero_act8_pack(x[a:b], q1, e1)
        z.zero_act8_unpack(q1, e1, o1)
        assert torch.equal(q[a:b], q1) and torch.equal(e[a:b], e1) and torch.equal(out[a:b], o1)
    eq, ee = act8(f64(x[-300:]))
    assert np.array_equal(q[-300:].cpu().numpy(), eq) and np.array_equal(e[-300:].cpu().numpy(), ee)


# ------------------------------------------------------------------ emitted values
@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("flags", [z.ACC_EMIT_BF16, z.ACC_EMIT_BF16 | z.ACC_NO_STORE,
                                   z.ACC_OVERWRITE | z.ACC_EMIT_BF16 | z.ACC_NO_STORE])
@pytest.mark.parametrize("vocab,cols,n,kind", [
    (1, 1, 1, "uniform"), (5, 4, 64, "same"), (3, 130, 1000, "uniform"), (300_000, 3, 5000, "skewed"),
    (50257, 16, 3000, "skewed"), (100, 1000, 129, "same"), (257, 4100, 64, "holes"),
    (2, 8, 20000, "uniform"), (7, 1030, 513, "same"), (40, 2050, 511, "skewed")])
def test_emb_grad_emits_what_it_sums(dtype, flags, vocab, cols, n, kind):
    """Sums of small integers: the emitted value is the exact sum, rounded once
    (integers up to 256 not at all), and nothing else is written."""
    L, pl = layout(vocab * cols, n % 2 == 1 and vocab * cols > 8)
    ids = some_ids(kind, n, vocab, n)
    dy = small_ints(n, n, cols, dtype=dtype)
    f = Flat(L, pl, vocab * cols, DEV, ints=True)
    z.zero_embedding_grad(L, 1, torch.from_numpy(ids.astype(np.int32)).to(DEV), dy, f.acc, 1.0,
                          flags, f.out)
    g, _ = emb_exact(ids, f64(dy), vocab)
    want = (0 if flags & z.ACC_OVERWRITE else f.acc0[f.pos]) + g
    assert torch.equal(f.out[torch.from_numpy(f.pos).to(DEV)].cpu(), torch.from_numpy(want).float().to(BF16))
    f.check(g, np.zeros(g.size), 1.0, flags, kind)


# ------------------------------------------------------------------ calls at the same time
class Work:
    """One micro-batch through all calls, with its own inputs, outputs and
    workspaces; results() of two passes have to be the same bits."""

    def __init__(self, seed, tokens, d, o, vocab):
        g = torch.Generator(device=DEV).manual_seed(seed)
        real = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF16)  # noqa: E731
        self.L = L = z.Layout([vocab * d, d, o * d], 0, 4, 0)
        self.ids = torch.randint(-1, vocab, (tokens,), generator=g, device=DEV)
        self.ids[: tokens // 4] = 3
        self.params, self.res, self.dout = real(L.padded), real(tokens, d), real(tokens, o)
        new = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype, device=DEV)  # noqa: E731
        self.x, self.h, self.y, self.dx, self.v = (new(tokens, d) for _ in range(5))
        self.rstd = new(tokens, dtype=torch.float32)
        self.acc, self.out = new(L.padded, dtype=torch.float32), new(L.padded)
        (self.q, self.e), lib = codes_like(tokens, d), z.load()
        flags = z.ACC_OVERWRITE | z.ACC_EMIT_BF16
        self.ws = [torch.empty(k + 16, dtype=torch.uint8, device=DEV) for k in (
            lib.zero_linear_grad_workspace(L.handle, 2, 0, o, d, tokens),
            lib.zero_rms_norm_grad_workspace(L.handle, 1, tokens),
            lib.zero_embedding_grad_workspace(L.handle, 0, d, tokens, flags))]
        self.flags = flags

    def run(self, stream=None):
        L, kw = self.L, {"stream": stream}
        z.zero_embedding_lookup(L, 0, self.params, self.ids, self.x, 2.0, **kw)
        z.zero_rms_norm(L, 1, self.params, self.x, self.res, 1e-5, self.h, self.rstd, self.q, self.e,
                        self.y, **kw)
        z.zero_act8_unpack(self.q, self.e, self.v, **kw)
        z.zero_linear_grad(L, 2, self.dout, self.q, self.e, self.acc, 0.5, self.flags, self.out,
                           workspace=self.ws[0], **kw)
        z.zero_rms_norm_grad(L, 1, self.params, self.v, self.res, self.h, self.rstd, self.dx, self.acc,
                             0.5, self.flags, self.out, workspace=self.ws[1], **kw)
        z.zero_embedding_grad(L, 0, self.ids, self.dx, self.acc, 0.5, self.flags, self.out,
                              workspace=self.ws[2], **kw)

    def results(self):
        return [t.clone() for t in (self.x, self.h, self.y, self.dx, self.v, self.rstd, self.acc,
                                    self.out, self.q, self.e)]

    def clear(self):
        for t in (self.x, self.h, self.y, self.dx, self.v, self.rstd, self.acc, self.out, self.q, self.e,
                  *self.ws):
            t.zero_()


def works():
    w = [Work(1, 700, 260, 300, 500), Work(2, 17_000, 136, 520, 300), Work(3, 3000, 1032, 264, 2000)]
    for one in w:
        one.run()
    torch.cuda.synchronize()
    return w, [one.results() for one in w]


def same(w, want):
    torch.cuda.synchronize()
    for k, (one, exp) in enumerate(zip(w, want)):
        for j, (a, b) in enumerate(zip(one.results(), exp)):
            assert torch.equal(a, b), f"micro-batch {k}, result {j}"


def test_calls_on_several_streams_at_once():
    w, want = works()
    streams = [torch.cuda.Stream() for _ in w]
    for turn in range(3):
        for one in w:
            one.clear()
        torch.cuda.synchronize()
        for _ in range(4):
            for one, s in zip(w, streams):
                one.run(s)
        same(w, want)


def test_calls_from_several_host_threads_at_once():
    w, want = works()
    for one in w:
        one.clear()
    torch.cuda.synchronize()
    errors = []

    def work(one):
        try:
            s = torch.cuda.Stream()
            for _ in range(6):
                one.run(s)
            s.synchronize()
        except Exception as e:                         # reported by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(one,)) for one in w]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    same(w, want)


def test_captured_graphs_replayed_at_once():
    """Each with its own workspaces, on streams of their own, with eager work
    between the replays."""
    w, want = works()
    graphs = []
    for one in w:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            one.run()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in w]
    for turn in range(4):
        for one in w:
            one.clear()
        torch.cuda.synchronize()
        for _ in range(2):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        same(w, want)
        torch.randn(1000, device=DEV).sum().item()     # the program's own work between


# ------------------------------------------------------------------ very large weights
@pytest.mark.parametrize("tr", [False, True])
def test_linear_grad_of_a_weight_beyond_32_bits(tr):
    """5.0e9 elements, 393216 tiles."""
    tokens, o, i = 3, 300, 1 << 24
    L = z.Layout([o * i], 0, 1, 0)
    g = torch.Generator(device=DEV).manual_seed(1)
    dy = torch.randint(-3, 4, (tokens, o), generator=g, device=DEV).to(BF16)
    x = torch.randint(-8, 9, (tokens, i), generator=g, device=DEV).to(BF16)
    q, e = codes_like(tokens, i)
    z.zero_act8_pack(x, q, e)
    acc = torch.ones(L.padded, device=DEV)
    z.zero_linear_grad(L, 0, dy, q, e, acc, 2.0, transposed=tr)
    dw = acc[:o * i].view(i, o) if tr else acc[:o * i].view(o, i)
    for k in range(0, i, 1 << 20):
        part = dy.float().t().contiguous() @ x[:, k:k + (1 << 20)].float() * 2 + 1   # small integers
        assert torch.equal(dw[k:k + (1 << 20)].t() if tr else dw[:, k:k + (1 << 20)], part)


# ------------------------------------------------------------------ calls that the header allows
@pytest.mark.parametrize("gaps", [False, True])
def test_emission_without_an_accumulator(gaps):
    """OVERWRITE with NO_STORE needs none."""
    flags = z.ACC_OVERWRITE | z.ACC_EMIT_BF16 | z.ACC_NO_STORE
    for cols, n in ((37, 700), (260, 700), (260, 0)):
        vocab = 90
        L, pl = layout(vocab * cols, gaps)
        ids, dy = some_ids("skewed", n, vocab, 1), small_ints(1, n, cols)
        f = Flat(L, pl, vocab * cols, DEV, ints=True)
        z.zero_embedding_grad(L, 1, torch.from_numpy(ids).to(DEV), dy, None, 0.5, flags, f.out)
        g, _ = emb_exact(ids, f64(dy), vocab)
        f.check(g, np.zeros(g.size), 0.5, flags, f"table {cols} {n}")
    rows, cols = 50, 300
    L, pl = layout(cols, gaps)
    dy, h = small_ints(2, rows, cols), small_ints(3, rows, cols)
    f, r, dx = Flat(L, pl, cols, DEV), torch.ones(rows, device=DEV), torch.empty(rows, cols, dtype=BF16, device=DEV)
    z.zero_rms_norm_grad(L, 1, torch.ones(L.padded, dtype=BF16, device=DEV), dy, None, h, r, dx, None, 0.5,
                         flags, f.out)
    f.check((f64(dy) * f64(h)).sum(0), np.zeros(cols), 0.5, flags, "norm")
    tokens, o, i = 300, 70, 130
    L, pl = layout(o * i, gaps)
    dy, x, (q, e) = small_ints(4, tokens, o), small_ints(5, tokens, i), codes_like(tokens, i)
    z.zero_act8_pack(x, q, e)
    f = Flat(L, pl, o * i, DEV)
    z.zero_linear_grad(L, 1, dy, q, e, None, 0.5, flags, f.out)
    f.check((f64(dy).T @ f64(x)).reshape(-1), np.zeros(o * i), 0.5, flags, "linear")


@pytest.mark.parametrize("flags", [0, z.ACC_OVERWRITE | z.ACC_EMIT_BF16])
@pytest.mark.parametrize("cols,n", [(7, 300), (7, 900), (264, 900)])
def test_table_and_norm_of_a_per_parameter_layout(cols, n, flags):
    """Each tensor in a slot of its own, padded behind its rows."""
    vocab = 61
    L, pl = layout(vocab * cols, False, dim0_rows=vocab)
    ids, dy = some_ids("holes", n, vocab, 2), small_ints(1, n, cols)
    idt, params = torch.from_numpy(ids).to(DEV), small_ints(6, L.padded)
    f = Flat(L, pl, vocab * cols, DEV, ints=True)
    z.zero_embedding_grad(L, 1, idt, dy, f.acc, 1.0, flags, f.out)
    g, _ = emb_exact(ids, f64(dy), vocab)
    f.check(g, np.zeros(g.size), 1.0, flags, "table")
    out = torch.empty(n, cols, dtype=torch.float32, device=DEV)
    z.zero_embedding_lookup(L, 1, params, idt, out, 0.5)
    rows = f64(params)[f.pos].reshape(vocab, cols)
    real = (ids >= 0) & (ids < vocab)
    assert np.array_equal(f64(out), np.where(real[:, None], rows[np.clip(ids, 0, vocab - 1)] * 0.5, 0.0))
    L, pl = layout(cols, False, dim0_rows=cols)
    f, h, r = Flat(L, pl, cols, DEV, ints=True), small_ints(7, n, cols), torch.ones(n, device=DEV)
    z.zero_rms_norm_grad(L, 1, torch.ones(L.padded, dtype=BF16, device=DEV), dy, None, h, r,
                         torch.empty(n, cols, dtype=BF16, device=DEV), f.acc, 1.0, flags, f.out)
    f.check((f64(dy) * f64(h)).sum(0), np.zeros(cols), 1.0, flags, "norm")


def test_an_empty_table_has_no_tokens():
    L = z.Layout([0, 40], 0, 4, 0)
    params, acc = torch.ones(L.padded, dtype=BF16, device=DEV), torch.ones(L.padded, device=DEV)
    ids = torch.tensor([0, -1, 5], device=DEV)
    out = torch.full((3, 8), 7.0, dtype=BF16, device=DEV)
    z.zero_embedding_lookup(L, 0, params, ids, out)
    assert not out.any()
    z.zero_embedding_grad(L, 0, ids, out, acc, 1.0, z.ACC_OVERWRITE)
    assert (acc == 1).all()


@pytest.mark.parametrize("n,flags", [(300, 0), (900, 0), (20_000, 0), (900, z.ACC_OVERWRITE)])
@pytest.mark.parametrize("cols", [37, 260])
@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_what_lies_in_places_without_a_token_is_not_used(n, flags, cols, dtype):
    """NaN and infinities there, and ids that are valid in their low bits only."""
    vocab = 50
    L, pl = layout(vocab * cols, False)
    ids = some_ids("uniform", n, vocab, 9)
    no = np.arange(n) % 3 == 1
    ids[no] = np.array([-1, 2 ** 32 + 4, -2 ** 63, 2 ** 63 - 1, vocab, -2 ** 32 + 7])[np.arange(no.sum()) % 6]
    dy = small_ints(1, n, cols, dtype=dtype)
    want, _ = emb_exact(np.where(no, -1, ids), f64(dy), vocab)
    bad = torch.from_numpy(no).to(DEV)
    dy[bad, ::2], dy[bad, 1::2] = float("nan"), float("inf")
    f = Flat(L, pl, vocab * cols, DEV, ints=True)
    z.zero_embedding_grad(L, 1, torch.from_numpy(ids).to(DEV), dy, f.acc, 1.0, flags)
    f.check(want, np.zeros(want.size), 1.0, flags, "gradient")
    params = torch.full((L.padded,), float("nan"), dtype=BF16, device=DEV)
    out = torch.full((n, cols), 7.0, dtype=dtype, device=DEV)
    z.zero_embedding_lookup(L, 1, params, torch.from_numpy(np.where(no, ids, -1)).to(DEV), out)
    assert not out.any()


def test_act8_of_the_smallest_and_largest_binary32_values():
    """Around the smallest code value 2^-126, halves of it among them, and up to
    the largest finite value, each in a block of its own."""
    k = np.arange(1, 65, dtype=np.float64)
    v = np.concatenate([k * 2.0 ** -130, (k + 0.5) * 2.0 ** -127, k * 2.0 ** -149,
                        (2.0 - 2.0 ** -23) * 2.0 ** np.arange(-126, 128), 1.75 * 2.0 ** np.arange(-126, 128),
                        (1.75 + 2.0 ** -22) * 2.0 ** np.arange(-126, 128)])
    v = np.concatenate([v, -v]).astype(np.float32)
    x = torch.from_numpy(v).view(-1, 1).to(DEV)
    (q, e), out = codes_like(v.size, 1), torch.empty(v.size, 1, device=DEV)
    z.zero_act8_pack(x, q, e)
    z.zero_act8_unpack(q, e, out)
    eq, ee = act8(v.astype(np.float64).reshape(-1, 1))
    assert np.array_equal(e.cpu().numpy(), ee) and np.array_equal(q.cpu().numpy(), eq)
    r = act8_values(eq, ee)
    r = np.where(np.abs(r) == 2.0 ** 128, np.copysign(np.inf, r), r)
    assert np.array_equal(f64(out), r)
