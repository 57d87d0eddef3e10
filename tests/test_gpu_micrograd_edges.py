"""The micro-batch operators on the GPU at the edges of their kernels: last,
partly filled groups of columns, turns of a block, addresses, calls at the same
time."""
import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_step_amd as z
from micrograd_ref import Flat, f64, layout
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
