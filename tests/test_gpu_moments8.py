"""The shard step with 8-bit moments on the GPU: every output equals the CPU
oracle's step on the values that the codes stand for, rounded to codes with
the same random bits."""
import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_step_amd as z
import moments8_ref as ref
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _free_gpu_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def at_offset(a, off):
    """A device copy whose memory begins `off` elements into an allocation."""
    t = torch.from_numpy(np.ascontiguousarray(a))
    buf = torch.zeros(t.numel() + off + 16, dtype=t.dtype, device=DEV)
    v = buf[off:off + t.numel()]
    v.copy_(t)
    return v


def layouts(numel, cap, n_d, rank, rows=None):
    if rows is None:
        return z.Layout(numel, cap, n_d, rank), oracle.plan(numel, cap, n_d)
    return z.Layout(numel, 0, n_d, rank, rows=rows), oracle.plan(numel, 0, n_d, rows=rows)


class Job:
    """A shard with contributions, and its twin in numpy."""

    def __init__(self, numel, cap, n_d, rank, f32=False, flat=False, slot=False, rows=None, off=0, seed=0):
        self.L, self.pl = layouts(numel, cap, n_d, rank, rows)
        self.flat, self.slot, self.rank, self.n_d = flat, slot, rank, n_d
        S, P = self.L.shard, self.L.padded
        assert S == self.pl.shard_len and self.L.moment_blocks == ref.slices(self.pl)[1]
        g = np.random.default_rng(seed)
        self.g = g
        self.idx = self.flat_places()
        self.f32, self.off = f32, off
        self.master = g.normal(size=S).astype(np.float32) * np.float32(0.02)
        m = (g.normal(size=S) * 1e-3).astype(np.float32)
        v = (g.normal(size=S) ** 2 * 1e-6 * 10.0 ** g.integers(-9, 1, S)).astype(np.float32)
        self.state = {"m": ref.encode_shard("m", self.pl, m), "v": ref.encode_shard("v", self.pl, v)}
        self.d_master = at_offset(self.master, off)
        self.moments = z.Moments8(*[at_offset(a, off) for k in ref.KINDS for a in self.state[k]])
        self.d_out = at_offset(np.full(P if slot else S, 7, np.int16), off)

    def flat_places(self):
        """Flat position of every shard element."""
        out = np.zeros(self.L.shard, np.int64)
        for (o, n, _), p in zip(ref.slices(self.pl)[0], self.pl.padded_off):
            out[o:o + n] = int(p) + self.rank * n + np.arange(n)
        return out

    def grads(self, scale=1e-3):
        n = self.L.padded if self.flat else self.L.shard
        gs = [(self.g.normal(size=n) * scale).astype(np.float32) for _ in range(self.n_d)]
        if not self.f32:
            gs = [oracle.round_bf16(x) for x in gs]
        dev = [at_offset(x if self.f32 else x.view(np.int16), self.off) for x in gs]
        return [x[self.idx] if self.flat else x for x in gs], dev

    def step(self, t, seed, grads=None, hp=None, **kw):
        host, dev = grads if grads is not None else self.grads()
        hp = hp or {}
        z.zero_shard_step_moments8(self.L, z.AdamW(**hp), t, dev, z.GRAD_FLAT if self.flat else z.GRAD_COMPACT,
                                   self.d_master, self.moments, self.d_out,
                                   z.OUT_AG_SLOT if self.slot else z.OUT_SHARD, seed, **kw)
        self.master, self.p, self.state = ref.step(self.pl, host, self.master, self.state, oracle.AdamW(**hp),
                                                   t, seed)

    def check(self):
        torch.cuda.synchronize()
        assert np.array_equal(self.d_master.cpu().numpy().view(np.uint32), self.master.view(np.uint32))
        out = self.d_out.cpu().numpy().view(np.uint16)
        if self.slot:
            rest = np.ones(out.size, bool)
            rest[self.idx] = False
            assert (out[rest] == 7).all()
            out = out[self.idx]
        assert np.array_equal(out, self.p)
        mom = self.moments
        for k, q, e in (("m", mom.exp_avg, mom.exp_avg_scales), ("v", mom.exp_avg_sq, mom.exp_avg_sq_scales)):
            assert np.array_equal(e.cpu().numpy(), self.state[k][1]), f"{k}: scales"
            assert np.array_equal(q.cpu().numpy(), self.state[k][0]), f"{k}: codes"


@pytest.mark.parametrize("n_d", [1, 2, 3, 4, 8, 16, 32, 64])
@pytest.mark.parametrize("f32", [False, True])
def test_rank_counts(n_d, f32):
    j = Job([700 * n_d + 3], 0, n_d, n_d - 1, f32=f32, flat=True, slot=True, seed=n_d)
    for t in (1, 2):
        j.step(t, 99)
        j.check()


@pytest.mark.parametrize("n", [1, 3, 4, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1027, 70001])
@pytest.mark.parametrize("off", [0, 1, 3])
def test_lengths_and_addresses(n, off):
    j = Job([2 * n - 1], 0, 2, 0, off=off, seed=n)
    j.step(5, 2 ** 63 + n)
    j.check()


@pytest.mark.parametrize("flat,slot", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("cap,n_d", [(100, 4), (1030, 3), (4096, 8), (513, 2)])
def test_buckets(flat, slot, cap, n_d):
    """Slices of any length: blocks begin anew in each."""
    j = Job([17, 6000, 5, 0, 2600], cap, n_d, 1, flat=flat, slot=slot, off=1, seed=cap)
    for t in (1, 2, 3):
        j.step(t, 7)
    j.check()


@pytest.mark.parametrize("flat,slot", [(False, False), (True, True)])
def test_a_tensor_each(flat, slot):
    """The per-parameter layout, more tensors than one launch takes, some of
    which this rank holds nothing of."""
    rows = [1 + (k * 7) % 23 for k in range(300)] + [0]
    numel = [r * (1 + (k * 13) % 61) for k, r in enumerate(rows)]
    j = Job(numel, 0, 4, 2, flat=flat, slot=slot, rows=rows, seed=3)
    for t in (1, 2):
        j.step(t, 1234)
    j.check()


def test_bucket_ranges_in_any_order_and_on_two_streams():
    a = Job([9000], 1000, 4, 3, flat=True, slot=True, seed=4)
    grads = a.grads()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for k, (b, e) in enumerate([(4, 7), (0, 1), (8, 9), (1, 4), (7, 8), (3, 3)]):
        z.zero_shard_step_moments8(a.L, z.AdamW(), 3, grads[1], z.GRAD_FLAT, a.d_master, a.moments, a.d_out,
                                   z.OUT_AG_SLOT, 5, bucket_begin=b, bucket_end=e, stream=side[k % 2])
    a.master, a.p, a.state = ref.step(a.pl, grads[0], a.master, a.state, oracle.AdamW(), 3, 5)
    a.check()


def test_dim0_bucket_range():
    rows = [8, 3, 20, 1, 9]
    numel = [8 * 33, 3 * 50, 20 * 7, 300, 9 * 129]
    a = Job(numel, 0, 4, 1, rows=rows, seed=4)
    host, dev = a.grads()
    before = a.d_master.clone()
    z.zero_shard_step_moments8(a.L, z.AdamW(), 3, dev, z.GRAD_COMPACT, a.d_master, a.moments, a.d_out,
                               z.OUT_SHARD, 5, bucket_begin=2, bucket_end=4)
    lo, hi = int(a.pl.shard_off[2]), int(a.pl.shard_off[4])
    kept = a.state
    th, p, st = ref.step(a.pl, host, a.master, a.state, oracle.AdamW(), 3, 5)
    got = a.d_master.cpu().numpy()
    assert np.array_equal(got[lo:hi], th[lo:hi])
    assert np.array_equal(got[:lo], before.cpu().numpy()[:lo]) and np.array_equal(got[hi:], before.cpu().numpy()[hi:])
    sl = ref.slices(a.pl)[0]
    s0, s1 = sl[2][2], sl[4][2]
    for k, q, e in (("m", a.moments.exp_avg, a.moments.exp_avg_scales),
                    ("v", a.moments.exp_avg_sq, a.moments.exp_avg_sq_scales)):
        q, e = q.cpu().numpy(), e.cpu().numpy()
        assert np.array_equal(q[lo:hi], st[k][0][lo:hi]) and np.array_equal(e[s0:s1], st[k][1][s0:s1])
        assert np.array_equal(q[:lo], kept[k][0][:lo]) and np.array_equal(q[hi:], kept[k][0][hi:])
        assert np.array_equal(e[:s0], kept[k][1][:s0]) and np.array_equal(e[s1:], kept[k][1][s1:])


def test_gradients_of_every_size():
    """Infinities, NaN, zeros, and magnitudes from subnormals to the largest."""
    j = Job([2048], 0, 1, 0, f32=True, seed=5)
    g = (j.g.normal(size=2048) * 10.0 ** j.g.integers(-44, 38, 2048)).astype(np.float32)
    g[:7] = [np.inf, -np.inf, np.nan, 0.0, -0.0, 1e-45, 3.4e38]
    g[256:384] = 0.0                                 # a block of nothing but decaying moments
    g[512:640] = np.inf                              # a block without a finite value
    j.step(1, 77, grads=([g], [at_offset(g, 0)]))
    torch.cuda.synchronize()
    mom, same = j.moments, lambda x, y: np.array_equal(x, y, equal_nan=True)  # noqa: E731
    assert same(j.d_master.cpu().numpy(), j.master)
    for k, q, e in (("m", mom.exp_avg, mom.exp_avg_scales), ("v", mom.exp_avg_sq, mom.exp_avg_sq_scales)):
        assert np.array_equal(e.cpu().numpy(), j.state[k][1])
        a, b = q.cpu().numpy(), j.state[k][0]
        nan = (b & 0x7F) == 0x7F if k == "m" else b == 255
        assert np.array_equal(a[~nan], b[~nan])
        assert (((a[nan] & 0x7F) == 0x7F) if k == "m" else (a[nan] == 255)).all()


def test_zero_bytes_are_zero_moments():
    j = Job([3000], 0, 2, 1, seed=6)
    j.moments = z.Moments8.zeros(j.L, DEV)
    n, b = j.L.shard, j.L.moment_blocks
    j.state = {k: (np.zeros(n, np.uint8), np.zeros(b, np.uint8)) for k in ref.KINDS}
    j.step(1, 0)
    j.check()


@pytest.mark.parametrize("rows", [None, [3, 40, 11]])
def test_pack_and_unpack(rows):
    numel = [3 * 50, 40 * 77, 11 * 260]
    L, pl = layouts(numel, 700, 4, 2, rows)
    S = L.shard
    g = np.random.default_rng(1)
    m = (g.normal(size=S) * 10.0 ** g.integers(-20, 20, S)).astype(np.float32)
    v = (g.normal(size=S) ** 2 * 10.0 ** g.integers(-30, 20, S)).astype(np.float32)
    m[3], m[200], v[4], v[300], v[5], v[301] = np.inf, np.nan, np.inf, np.nan, -1.0, -0.0
    mom = z.Moments8.zeros(L, DEV)
    z.zero_moments8_pack(L, at_offset(m, 1), at_offset(v, 3), mom)
    back = [torch.empty(S, dtype=torch.float32, device=DEV) for _ in range(2)]
    z.zero_moments8_unpack(L, mom, *back)
    v = np.where(v < 0, np.float32(0), v)
    for k, x, q, e, b in (("m", m, mom.exp_avg, mom.exp_avg_scales, back[0]),
                          ("v", v, mom.exp_avg_sq, mom.exp_avg_sq_scales, back[1])):
        codes, scales = ref.encode_shard(k, pl, x)
        nan = ~np.isfinite(x)
        q = q.cpu().numpy()
        assert np.array_equal(e.cpu().numpy(), scales)
        assert np.array_equal(q[~nan], codes[~nan])
        assert np.array_equal(b.cpu().numpy(), ref.decode_shard(k, pl, codes, scales), equal_nan=True)
        again = z.Moments8.zeros(L, DEV)
        z.zero_moments8_pack(L, *back, again)
        twice = [torch.empty_like(y) for y in back]
        z.zero_moments8_unpack(L, again, *twice)
        for y, w in zip(back, twice):
            assert np.array_equal(y.cpu().numpy(), w.cpu().numpy(), equal_nan=True)


def test_captured_and_replayed():
    j = Job([5000], 600, 2, 1, flat=True, slot=True, seed=8)
    grads = j.grads()
    eager = Job([5000], 600, 2, 1, flat=True, slot=True, seed=8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        z.zero_shard_step_moments8(j.L, z.AdamW(), 4, grads[1], z.GRAD_FLAT, j.d_master, j.moments, j.d_out,
                                   z.OUT_AG_SLOT, 11)
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        j.master, j.p, j.state = ref.step(j.pl, grads[0], j.master, j.state, oracle.AdamW(), 4, 11)
        eager.step(4, 11, grads=grads)              # eager work between the replays
        j.check()
        eager.check()


def test_a_shard_past_32_bits():
    """Elements past 2^32: their addresses, scale bytes and random bits."""
    n = (1 << 32) + 1000
    L = z.Layout([n], 0, 1, 0)
    new = lambda k, dtype: torch.zeros(k, dtype=dtype, device=DEV)  # noqa: E731
    master, grad, out = new(n, torch.float32), new(n, torch.bfloat16), new(n, torch.bfloat16)
    mom = z.Moments8(new(n, torch.uint8), new(L.moment_blocks, torch.uint8), new(n, torch.uint8),
                     new(L.moment_blocks, torch.uint8))
    lo = (1 << 32) - 128 * 9                        # the random bits' carry lies inside
    g = oracle.round_bf16((np.random.default_rng(2).normal(size=n - lo) * 1e-3).astype(np.float32))
    grad[lo:] = torch.from_numpy(g.view(np.int16)).view(torch.bfloat16).to(DEV)
    z.zero_shard_step_moments8(L, z.AdamW(), 1, [grad], z.GRAD_COMPACT, master, mom, out, z.OUT_SHARD, 3)
    m, v, th = (np.zeros(n - lo, np.float32) for _ in range(3))
    p, _ = oracle.shard_step([g], th, m, v, oracle.AdamW(), 1)
    h = ref.random_bits(3, 1, np.arange(lo, n))
    assert np.array_equal(master[lo:].cpu().numpy(), th)
    assert np.array_equal(out[lo:].view(torch.int16).cpu().numpy().view(np.uint16), p)
    for k, x, r, q, e in (("m", m, h & np.uint64(0xFFFF), mom.exp_avg, mom.exp_avg_scales),
                          ("v", v, h >> np.uint64(16), mom.exp_avg_sq, mom.exp_avg_sq_scales)):
        codes, scales = ref.encode(k, x, r)
        assert np.array_equal(q[lo:].cpu().numpy(), codes) and np.array_equal(e[lo // 128:].cpu().numpy(), scales)
    assert not bool(mom.exp_avg[:4096].any()) and not bool(master[(1 << 31):(1 << 31) + 4096].any())


def test_moments_keep_their_expected_value():
    """A moment that decays by less than half the distance of two codes a step
    still decays: after 500 steps without gradients the sum over 2^16 second
    moments is beta2^500 of what it was, within 5 standard deviations.  A
    step's rounding adds at most (step/2)^2 <= (v/32)^2 to an element's
    variance, so after k steps it is at most k * (v/32)^2 with v the first
    value (every later one is expected to be smaller, and E v^2 grows at most
    by (1 + 2^-10) a step): the sum's is 2^16 of that."""
    n, k, b2 = 1 << 16, 500, 0.999
    L = z.Layout([n], 0, 1, 0)
    mom = z.Moments8.zeros(L, DEV)
    v0 = torch.full((n,), 1.0e-6, dtype=torch.float32, device=DEV)
    zero = torch.zeros(n, dtype=torch.float32, device=DEV)
    z.zero_moments8_pack(L, zero, v0, mom)
    start, m, v = torch.empty_like(v0), torch.empty_like(v0), torch.empty_like(v0)
    z.zero_moments8_unpack(L, mom, m, start)
    grad, out, master = zero.bfloat16(), zero.bfloat16(), zero.clone()
    for t in range(1, k + 1):
        z.zero_shard_step_moments8(L, z.AdamW(beta2=b2), t, [grad], z.GRAD_COMPACT, master, mom, out,
                                   z.OUT_SHARD, 17)
    z.zero_moments8_unpack(L, mom, m, v)
    exp = float(start.double().sum()) * b2 ** k
    one = float(start[0])
    sigma = (n * k * (1 + 2.0 ** -10) ** k) ** 0.5 * one / 32
    assert abs(float(v.double().sum()) - exp) <= 5 * sigma
    assert 5 * sigma < 0.1 * exp and not bool(m.any())


def test_small_moments_stay_at_the_smallest_code():
    """Blocks of one large second moment, which a gradient of its root keeps where
    it is, and small ones without gradients.  Those of one smallest code stay
    there, those of three come down to it and no further; those of 1024 decay as
    expected, with the bound of the test above."""
    blocks, k, b2 = 512, 500, 0.999
    n, unit = 128 * blocks, 2.0 ** -18
    L = z.Layout([n], 0, 1, 0)
    mom = z.Moments8.zeros(L, DEV)
    v0 = torch.full((blocks, 128), 1024 * unit, dtype=torch.float32, device=DEV)
    v0[:, 0], v0[:, 1:43], v0[:, 43:85] = 1.0, unit, 3 * unit
    zero = torch.zeros(n, dtype=torch.float32, device=DEV)
    z.zero_moments8_pack(L, zero, v0.view(-1), mom)
    m, v = torch.empty_like(zero), torch.empty_like(v0)
    grad = torch.zeros(blocks, 128, dtype=torch.bfloat16, device=DEV)
    grad[:, 0] = 1.0
    out, master = zero.bfloat16(), zero.clone()
    for t in range(1, k + 1):
        z.zero_shard_step_moments8(L, z.AdamW(beta2=b2), t, [grad.view(-1)], z.GRAD_COMPACT, master, mom, out,
                                   z.OUT_SHARD, 19)
    z.zero_moments8_unpack(L, mom, m, v.view(-1))
    v = v.double()
    assert (v[:, 1:43] == unit).all()
    assert (v[:, 43:85] >= unit).all() and (v[:, 43:85] == unit).any()
    exp, count = 1024 * unit * b2 ** k, blocks * 43
    sigma = (count * k * (1 + 2.0 ** -10) ** k) ** 0.5 * 1024 * unit / 32
    assert abs(float(v[:, 85:].sum()) - count * exp) <= 5 * sigma and 5 * sigma < 0.1 * count * exp
    assert (v[:, 0] >= 1 - 2.0 ** -4).all()
