"""The operators of a training step run together on one rank's flat buffers: a
projection to queries, keys and values, their norms and rotation, the
projection back, a feed-forward layer with its activation, the way back through
all of them, and the step with 8-bit moments on what they accumulated.
"""
import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_step_amd as z
import moments8_ref as mref
import oracle
from micrograd_ref import f64
from test_gpu_micrograd import randn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32, F8, U8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.uint8
T, HQ, HK, D, FF = 150, 4, 2, 32, 200
DIM = HQ * D
WIDE = (HQ + 2 * HK) * D
EPS = 1e-6
NAMES = ["w_qkv", "b_qkv", "q_norm", "k_norm", "w_o", "w_up", "b_up", "w_down", "b_down"]
SHAPES = [(WIDE, DIM), (WIDE,), (D,), (D,), (DIM, DIM), (FF, DIM), (FF,), (FF, DIM), (DIM,)]
ID = {n: k for k, n in enumerate(NAMES)}


@pytest.fixture(autouse=True)
def _free_gpu_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


class Block:
    """Flat parameters, accumulator and everything that one micro-batch keeps."""

    def __init__(self, cap, n_d):
        self.numel = [int(np.prod(s)) for s in SHAPES]
        self.L = z.Layout(self.numel, cap, n_d, 0)
        self.pl = oracle.plan(self.numel, cap, n_d)
        x = np.arange(sum(self.numel))
        b = np.searchsorted(self.pl.stream_off, x, side="right") - 1
        place = torch.from_numpy(np.asarray(self.pl.padded_off)[b] + x - np.asarray(self.pl.stream_off)[b]).to(DEV)
        self.place = dict(zip(NAMES, place.split(self.numel)))
        self.params = torch.zeros(self.L.padded, dtype=BF16, device=DEV)
        for k, (n, s) in enumerate(zip(NAMES, SHAPES)):
            w = randn(k, *s) * (1.0 if len(s) == 1 else s[-1] ** -0.5)
            self.params[self.place[n]] = (w + 1 if "norm" in n else w).reshape(-1).to(BF16)
        self.acc = torch.zeros(self.L.padded, device=DEV)
        self.turn = z.Rotation(torch.arange(T, dtype=torch.int32, device=DEV),
                               100.0 ** (-torch.arange(D // 2, dtype=torch.float64, device=DEV) / (D // 2)))
        new = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype, device=DEV)  # noqa: E731
        self.x, self.dy, self.dk, self.dv = randn(20, T, DIM), randn(21, T, DIM), randn(22, T, HK, D), randn(23, T, HK * D)
        self.qkv, self.dqkv = new(T, WIDE), new(T, WIDE)
        self.q, self.k = new(T, HQ, D), new(T, HK, D)
        self.h, self.pre, self.u, self.y = new(T, DIM), new(T, FF), new(T, FF), new(T, DIM)
        self.dup, self.dh, self.da, self.dx = new(T, FF), new(T, DIM), new(T, DIM), new(T, DIM)
        self.codes = {n: (new(T, c, dtype=U8), new(T, -(-c // 128), dtype=U8))
                      for n, c in (("x", DIM), ("a", DIM), ("h", DIM), ("u", FF))}

    def heads(self, t):
        """Queries and keys of a token's row."""
        return t[:, :HQ * D].view(T, HQ, D), t[:, HQ * D:(HQ + HK) * D].view(T, HK, D)

    def forward(self):
        L, p = self.L, self.params
        z.zero_linear(L, ID["w_qkv"], p, self.x, self.qkv, bias=ID["b_qkv"])
        z.zero_head_norm_rotate(L, ID["q_norm"], ID["k_norm"], p, *self.heads(self.qkv), EPS, self.turn, self.q, self.k)
        a = self.q.view(T, DIM)                     # in the place of the attention over q and k
        z.zero_linear(L, ID["w_o"], p, a, self.h, res=self.x)
        z.zero_linear(L, ID["w_up"], p, self.h, self.u, bias=ID["b_up"], activation="gelu", pre=self.pre)
        z.zero_linear(L, ID["w_down"], p, self.u, self.y, bias=ID["b_down"], res=self.h, transposed=True)
        for n, t in (("x", self.x), ("a", a), ("h", self.h), ("u", self.u)):
            z.zero_act8_pack(t, *self.codes[n])

    def backward(self):
        L, p, acc = self.L, self.params, self.acc
        z.zero_bias_grad(L, ID["b_down"], self.dy, acc)
        z.zero_linear_grad(L, ID["w_down"], self.dy, *self.codes["u"], acc, transposed=True)
        z.zero_linear_input_grad(L, ID["w_down"], p, self.dy, self.dup, activation="gelu", pre=self.pre, transposed=True)
        z.zero_bias_grad(L, ID["b_up"], self.dup, acc)
        z.zero_linear_grad(L, ID["w_up"], self.dup, *self.codes["h"], acc)
        z.zero_linear_input_grad(L, ID["w_up"], p, self.dup, self.dh, add=self.dy)
        z.zero_linear_grad(L, ID["w_o"], self.dh, *self.codes["a"], acc)
        z.zero_linear_input_grad(L, ID["w_o"], p, self.dh, self.da)
        self.dqkv[:, (HQ + HK) * D:].copy_(self.dv)
        z.zero_head_norm_rotate_grad(L, ID["q_norm"], ID["k_norm"], p, self.da.view(T, HQ, D), self.dk,
                                     *self.heads(self.qkv), EPS, self.turn, *self.heads(self.dqkv), acc)
        z.zero_bias_grad(L, ID["b_qkv"], self.dqkv, acc)
        z.zero_linear_grad(L, ID["w_qkv"], self.dqkv, *self.codes["x"], acc)
        z.zero_linear_input_grad(L, ID["w_qkv"], p, self.dqkv, self.dx, add=self.dh)

    def reference(self):
        """Output and gradients by automatic differentiation in 64 bits, what is
        stored rounded to bf16 where the calls round it."""
        w = {n: self.params[self.place[n]].double().view(*s).requires_grad_() for n, s in zip(NAMES, SHAPES)}
        x = self.x.double().requires_grad_()

        def stored(t):
            """Rounded as stored; the rounding counts as the identity."""
            return t + (t.float().bfloat16().double() - t).detach()
        qkv = stored(x @ w["w_qkv"].t() + w["b_qkv"])
        angle = (torch.arange(T, device=DEV).double()[:, None] * self.turn.freqs)[:, None, :]
        out = []
        for t, g in zip(self.heads(qkv), ("q_norm", "k_norm")):
            u = t / (t.square().mean(2, keepdim=True) + EPS).sqrt() * w[g]
            a, b = u[..., :D // 2], u[..., D // 2:]
            out.append(stored(torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], 2)))
        h = stored(out[0].reshape(T, DIM) @ w["w_o"].t() + x)
        u = h @ w["w_up"].t() + w["b_up"]
        u = stored(u * torch.special.ndtr(u))
        y = stored(u @ w["w_down"] + w["b_down"] + h)
        loss = (y * self.dy.double()).sum() + (out[1] * self.dk.double()).sum() + (qkv[:, (HQ + HK) * D:] * self.dv.double()).sum()
        loss.backward()
        return y.detach(), {"x": x.grad, **{n: w[n].grad.reshape(-1) for n in NAMES}}


@pytest.mark.parametrize("cap,n_d", [(0, 4), (20011, 4)])
def test_forward_backward_and_step(cap, n_d):
    """Whole buckets, and buckets whose padding falls inside weights."""
    b = Block(cap, n_d)
    b.forward()
    b.backward()
    y, grads = b.reference()
    # Forward and backward store ten tensors one after another; each stored
    # value is off by half a step, 2^-8 of itself, at most against the same value
    # unrounded, and by one more where the two sides round apart; the weights'
    # gradients read inputs in e4m3, 2^-4 of a value off at most.  The maps
    # between are random: errors pass through them with the gain of the values.
    # Norms of errors add up to ten times 2^-7, and 2^-4 for e4m3.
    near = lambda got, exp, tol: float((got.double() - exp).norm() / exp.norm()) <= tol  # noqa: E731
    assert near(b.y, y, 10 * 2.0 ** -7)
    assert near(b.dx, grads["x"], 10 * 2.0 ** -7)
    for n in NAMES:
        assert near(b.acc[b.place[n]], grads[n], 10 * 2.0 ** -7 + (2.0 ** -4 if n.startswith("w_") else 0)), n
    rest = torch.ones(b.L.padded, dtype=torch.bool, device=DEV)
    for n in NAMES:
        rest[b.place[n]] = False
    assert not bool(b.acc[rest].any())

    # every rank steps its shard on all ranks' accumulators, whole flat buffers
    accs = [b.acc * s for s in np.linspace(0.5, 1.5, n_d)]
    host = [a.cpu().numpy() for a in accs]
    shards, expected = [], np.zeros(b.L.padded, np.uint16)
    for r in range(n_d):
        L = z.Layout(b.numel, cap, n_d, r)
        idx = np.zeros(L.shard, np.int64)
        for (o, n, _), padded in zip(mref.slices(b.pl)[0], b.pl.padded_off):
            idx[o:o + n] = int(padded) + r * n + np.arange(n)
        master = f64(b.params)[idx].astype(np.float32)
        d_master, mom = torch.from_numpy(master).to(DEV), z.Moments8.zeros(L, DEV)
        out = torch.zeros(L.shard, dtype=BF16, device=DEV)
        state = {k: (np.zeros(L.shard, np.uint8), np.zeros(L.moment_blocks, np.uint8)) for k in mref.KINDS}
        for t in (1, 2):
            z.zero_shard_step_moments8(L, z.AdamW(), t, accs, z.GRAD_FLAT, d_master, mom, out, z.OUT_SHARD, seed=r)
            master, p, state = mref.step(b.pl, [h[idx] for h in host], master, state, oracle.AdamW(), t, r)
        assert np.array_equal(d_master.cpu().numpy(), master)
        assert np.array_equal(mom.exp_avg_sq.cpu().numpy(), state["v"][0])
        shards.append(out)
        expected[idx] = p
    z.zero_gather_params(b.L, shards, b.params)
    assert np.array_equal(b.params.view(torch.int16).cpu().numpy().view(np.uint16), expected)
    b.forward()                                     # and the next step's forward pass reads them
    assert bool(torch.isfinite(b.y).all())


def test_captured_with_an_eager_one_beside():
    """Forward and backward passes captured and replayed, each time equal to
    eager ones of another block's buffers."""
    a, b = Block(20011, 4), Block(20011, 4)
    a.forward()                                     # builds nothing up: the calls keep no state
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.forward()
        a.backward()
    for _ in range(3):
        a.acc.zero_()
        g.replay()
        b.acc.zero_()
        b.forward()
        b.backward()
        torch.cuda.synchronize()
        assert torch.equal(a.acc, b.acc) and torch.equal(a.dx, b.dx) and torch.equal(a.y, b.y)
