"""Cases and plain forms of the operators that turn a micro-batch into parameter gradients.

Six calls around the rank's flat (padded bucket) buffers:

  lookup      rows of an embedding table that lies in the gathered parameter buffer, scaled
  emb_grad    the table's gradient, summed by token, into the fp32 accumulator (or emitted in bf16)
  norm        root-mean-square norm with the residual's addition and an 8-bit output with scales
  norm_grad   its backward pass, the weight's gradient into the fp32 accumulator
  act8        an activation checkpoint in 8 bits, written and read back
  linear_grad a linear weight's gradient from the output gradient and an 8-bit checkpoint

8-bit format: e4m3 codes, one power-of-two scale (its biased exponent, a byte) for every 128
columns of a row.  With own = False everything is elementary torch in 32 bits.
"""
import torch

own = False

DEV = "cuda"
CAP = 25 * 1024 * 1024 // 2     # elements of a 25 MiB bf16 bucket, as the workloads cut them
N_D = 8
EPS = 1e-5


def listed():
    return [
        # a GPT-2 context of one sequence
        {"name": "lookup gpt2 1024", "op": "lookup", "t": 1024, "v": 50257, "d": 768},
        # four sequences of 4096 tokens, the Llama-70B table
        {"name": "lookup llama70b 16384", "op": "lookup", "t": 16384, "v": 128256, "d": 8192},
        # the last micro-batch of a GPT-2 step: the whole table's gradient is emitted in bf16
        {"name": "emb_grad gpt2 emit", "op": "emb_grad", "t": 1000, "v": 50257, "d": 768, "emit": True},
        # an earlier micro-batch, four sequences of 4096 tokens, the Llama-3-8B table
        {"name": "emb_grad llama8b 16384", "op": "emb_grad", "t": 16384, "v": 128256, "d": 4096, "emit": False},
        # a short, ragged batch at GPT-2's width
        {"name": "norm 333x768", "op": "norm", "t": 333, "d": 768},
        # a Llama-70B block's norm over 16384 tokens
        {"name": "norm 16384x8192", "op": "norm", "t": 16384, "d": 8192},
        {"name": "norm_grad 333x768", "op": "norm_grad", "t": 333, "d": 768},
        # a Llama-3-8B block's norm
        {"name": "norm_grad 16384x4096", "op": "norm_grad", "t": 16384, "d": 4096},
        # one sequence kept in fp32, at an odd width
        {"name": "act8 fp32 1000x770", "op": "act8", "t": 1000, "d": 770, "f32": True},
        # the input of Llama-3-8B's down projection
        {"name": "act8 8192x14336", "op": "act8", "t": 8192, "d": 14336, "f32": False},
        # Llama-3-8B's key projection, one ragged sequence: few output tiles, a long sum
        {"name": "linear_grad 4000x1024x4096", "op": "linear_grad", "t": 4000, "o": 1024, "i": 4096, "tr": False},
        # Llama-3-8B's gate projection over 16384 tokens
        {"name": "linear_grad 16384x14336x4096", "op": "linear_grad", "t": 16384, "o": 14336, "i": 4096, "tr": False},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _width(rng, hi):
    """A row's length: half of the time a multiple of 128, else anything."""
    d = _log(rng, 64, hi)
    return max(128, d // 128 * 128) if rng.random() < 0.5 else d


def draw(rng):
    op = rng.choice(["lookup", "emb_grad", "norm", "norm_grad", "act8", "linear_grad"])
    if op == "lookup":
        return {"op": op, "t": _log(rng, 1, 16384), "v": _log(rng, 500, 128256), "d": _width(rng, 8192)}
    if op == "emb_grad":
        emit = rng.random() < 0.4
        v = _log(rng, 500, 50257 if emit else 128256)
        return {"op": op, "t": _log(rng, 1, 16384), "v": v, "d": _width(rng, 768 if emit else 4096), "emit": emit}
    if op == "norm":
        return {"op": op, "t": _log(rng, 1, 16384), "d": _width(rng, 8192)}
    if op == "norm_grad":
        return {"op": op, "t": _log(rng, 1, 16384), "d": _width(rng, 4096)}
    if op == "act8":
        return {"op": op, "t": _log(rng, 1, 8192), "d": _width(rng, 14336), "f32": rng.random() < 0.3}
    return {"op": op, "t": _log(rng, 16, 16384), "o": _width(rng, 14336), "i": _width(rng, 4096),
            "tr": rng.random() < 0.3}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFFFFFF)
    return g


def _randn(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device=DEV, dtype=dtype) * scale)


def _padded(n):
    """Length of the flat buffer of one tensor of n elements (its last bucket padded to the ranks)."""
    return -(-n // N_D) * N_D


def _ids(g, t, v):
    """Token ids, few of them frequent and most rare; a sixteenth of the places hold no token (-1)."""
    u = torch.rand(t, generator=g, device=DEV, dtype=torch.float64)
    ids = (u * u * u * v).to(torch.int64).clamp_(max=v - 1)
    ids = (ids * 7919) % v if v % 7919 else ids
    return torch.where(torch.rand(t, generator=g, device=DEV) < 1 / 16, -1, ids)


def _activations(g, t, d, dtype=torch.bfloat16):
    """Activations: normal, with some columns far larger than the rest."""
    x = torch.randn(t, d, generator=g, device=DEV, dtype=dtype)
    big = 1 + 30 * (torch.rand(d, generator=g, device=DEV) < 0.01).to(dtype)
    return x.mul_(big)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case)
    t = case["t"]
    if op == "lookup":
        v, d = case["v"], case["d"]
        s["params"] = _randn(g, _padded(v * d), scale=0.02)
        s["ids"] = _ids(g, t, v)
        s["scale"] = d ** 0.5
    elif op == "emb_grad":
        v, d = case["v"], case["d"]
        s["ids"] = _ids(g, t, v)
        s["dy"] = _randn(g, t, d, scale=1e-3)
        s["acc"] = _randn(g, _padded(v * d), scale=1e-3, dtype=torch.float32)
        s["scale"] = 0.25
        if case["emit"]:
            s["out"] = torch.zeros(_padded(v * d), dtype=torch.bfloat16, device=DEV)
    elif op in ("norm", "norm_grad"):
        d = case["d"]
        s["params"] = 1 + _randn(g, _padded(d), scale=0.1)
        if op == "norm":
            s["x"], s["res"] = _randn(g, t, d), _activations(g, t, d)
        else:
            s["h"] = _activations(g, t, d)
            s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + EPS).float()
            s["dy"], s["dh"] = _randn(g, t, d, scale=1e-2), _randn(g, t, d, scale=1e-2)
            s["acc"] = _randn(g, _padded(d), dtype=torch.float32)
            s["scale"] = 0.25
    elif op == "act8":
        s["x"] = _activations(g, t, case["d"], torch.float32 if case["f32"] else torch.bfloat16)
    else:
        o, i = case["o"], case["i"]
        s["q"], s["e"] = _quantise(_activations(g, t, i).float())
        s["dy"] = _randn(g, t, o, scale=1e-3)
        s["acc"] = _randn(g, _padded(o * i), scale=1e-2, dtype=torch.float32)
        s["scale"] = 0.25
    return s


# ------------------------------------------------------------------ plain forms
def _quantise(x):
    """(codes, scale bytes) of the rows of x: the scale is the smallest power of two, its byte
    at least 10, by which the block's largest value comes to 448 at most."""
    t, d = x.shape
    nb = -(-d // 128)
    xp = torch.nn.functional.pad(x, (0, nb * 128 - d)).view(t, nb, 128)
    m, k = torch.frexp(xp.abs().amax(2))                     # amax = m 2^k, 1/2 <= m < 1
    e = (127 + k - 9 + (m > 0.875).to(k.dtype)).clamp_(min=10)
    q = torch.ldexp(xp, (127 - e).unsqueeze(2)).to(torch.float8_e4m3fn)
    return q.view(t, nb * 128)[:, :d].contiguous(), e.to(torch.uint8)


def _values(q, e, dtype=torch.float32):
    t, d = q.shape
    x = torch.nn.functional.pad(q.to(dtype), (0, e.shape[1] * 128 - d)).view(t, -1, 128)
    return torch.ldexp(x, (e.to(torch.int32) - 127).unsqueeze(2)).view(t, -1)[:, :d]


def _plain(s):
    op = s["op"]
    if op == "lookup":
        v, d, ids = s["v"], s["d"], s["ids"]
        real = ((ids >= 0) & (ids < v)).unsqueeze(1)
        rows = s["params"][:v * d].view(v, d)[ids.clamp(0, v - 1)].float() * s["scale"]
        return torch.where(real, rows, 0.0).to(torch.bfloat16)
    if op == "emb_grad":
        v, d, ids = s["v"], s["d"], s["ids"]
        real = ((ids >= 0) & (ids < v)).unsqueeze(1)
        rows = torch.where(real, s["dy"].float() * s["scale"], 0.0)
        if s["emit"]:
            a = s["acc"][:v * d].view(v, d).index_add(0, ids.clamp(0, v - 1), rows)
            s["out"][:v * d] = a.view(-1).to(torch.bfloat16)
            return s["out"]
        s["acc"][:v * d].view(v, d).index_add_(0, ids.clamp(0, v - 1), rows)
        return s["acc"]
    if op == "norm":
        w = s["params"][:s["d"]].float()
        h = (s["x"].float() + s["res"].float()).to(torch.bfloat16)
        hf = h.float()
        rstd = 1 / torch.sqrt(hf.square().mean(1) + EPS)
        q, e = _quantise(hf * rstd.unsqueeze(1) * w)
        return {"h": h, "rstd": rstd, "y": _values(q, e).to(torch.bfloat16)}
    if op == "norm_grad":
        d = s["d"]
        w, h, r, dy = s["params"][:d].float(), s["h"].float(), s["rstd"].unsqueeze(1), s["dy"].float()
        gy = dy * w
        c = (gy * h).mean(1, keepdim=True) * r * r
        dx = s["dh"].float() + r * (gy - c * h)
        s["acc"][:d] += s["scale"] * (dy * h * r).sum(0)
        return {"dx": dx.to(torch.bfloat16), "acc": s["acc"]}
    if op == "act8":
        return _values(*_quantise(s["x"].float())).to(torch.bfloat16)
    o, i = s["o"], s["i"]
    x, dy = _values(s["q"], s["e"]), s["dy"].float()
    g = x.t() @ dy if s["tr"] else dy.t() @ x
    s["acc"][:o * i] += s["scale"] * g.reshape(-1)
    return s["acc"]


def _layout(z, s, numel):
    """The layout that a program keeps next to its buffers."""
    if "layout" not in s:
        s["layout"] = z.Layout([numel], CAP, N_D, 0)
    return s["layout"]


def _own(s):
    import fsdp_sharded_optimizer_step_amd as z
    op, t = s["op"], s["t"]
    new = lambda *shape, dtype=torch.bfloat16: torch.empty(*shape, dtype=dtype, device=DEV)  # noqa: E731
    if op == "lookup":
        L = _layout(z, s, s["v"] * s["d"])
        out = new(t, s["d"])
        z.zero_embedding_lookup(L, 0, s["params"], s["ids"], out, scale=s["scale"])
        return out
    if op == "emb_grad":
        L = _layout(z, s, s["v"] * s["d"])
        if s["emit"]:
            z.zero_embedding_grad(L, 0, s["ids"], s["dy"], s["acc"], s["scale"],
                                  z.ACC_EMIT_BF16 | z.ACC_NO_STORE, s["out"])
            return s["out"]
        z.zero_embedding_grad(L, 0, s["ids"], s["dy"], s["acc"], s["scale"])
        return s["acc"]
    if op in ("norm", "norm_grad"):
        d = s["d"]
        L = _layout(z, s, d)
        if op == "norm":
            h, y, rstd = new(t, d), new(t, d), new(t, dtype=torch.float32)
            q, e = new(t, d, dtype=torch.float8_e4m3fn), new(t, -(-d // 128), dtype=torch.uint8)
            z.zero_rms_norm(L, 0, s["params"], s["x"], s["res"], EPS, h, rstd, q, e, y)
            return {"h": h, "rstd": rstd, "y": y}
        dx = new(t, d)
        z.zero_rms_norm_grad(L, 0, s["params"], s["dy"], s["dh"], s["h"], s["rstd"], dx, s["acc"],
                             s["scale"])
        return {"dx": dx, "acc": s["acc"]}
    if op == "act8":
        d = s["d"]
        q, e = new(t, d, dtype=torch.float8_e4m3fn), new(t, -(-d // 128), dtype=torch.uint8)
        z.zero_act8_pack(s["x"], q, e)
        out = new(t, d)
        z.zero_act8_unpack(q, e, out)
        return out
    L = _layout(z, s, s["o"] * s["i"])
    z.zero_linear_grad(L, 0, s["dy"], s["q"], s["e"], s["acc"], s["scale"], transposed=s["tr"])
    return s["acc"]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ work
def _distinct(t, v):
    """Expected number of distinct ids among t draws of _ids()."""
    edge = torch.linspace(0, 1, v + 1, dtype=torch.float64) ** (1 / 3)
    p = (edge[1:] - edge[:-1]) * (15 / 16)
    return float((1 - (1 - p) ** t).sum())


def work(case):
    op, t = case["op"], case["t"]
    if op == "lookup":
        n = case["d"] * 2
        return {"bytes": t * 8 + _distinct(t, case["v"]) * n + t * n, "flops": t * case["d"]}
    if op == "emb_grad":
        v, d = case["v"], case["d"]
        n = t * 8 + t * d * 2 * 15 / 16
        n += v * d * 6 if case["emit"] else _distinct(t, v) * d * 8
        return {"bytes": n, "flops": 2 * t * d}
    if op == "norm":
        n = t * case["d"]
        return {"bytes": n * (2 + 2 + 2 + 1 + 2) + t * 4 + n / 128, "flops": 8 * n}
    if op == "norm_grad":
        n = t * case["d"]
        return {"bytes": n * 8 + t * 4 + case["d"] * 10, "flops": 12 * n}
    if op == "act8":
        n = t * case["d"]
        return {"bytes": n * ((4 if case["f32"] else 2) + 1 + 1 + 2) + n / 64, "flops": 6 * n}
    o, i = case["o"], case["i"]
    return {"bytes": t * o * 2 + t * i * (1 + 1 / 128) + o * i * 8, "flops": 2 * t * o * i}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_act8(x):
    """Values that the 8-bit form of the rows of x (64 bits) stands for, from the definition:
    the nearest multiple of the code's step, ties to the even multiple."""
    t, d = x.shape
    out = torch.empty_like(x)
    for b in range(0, d, 128):
        blk = x[:, b:b + 128]
        a = blk.abs().amax(1, keepdim=True)
        k = torch.floor(torch.log2(a.clamp(min=2.0 ** -300)))
        k = torch.where(torch.exp2(k) > a, k - 1, k)
        k = torch.where(torch.exp2(k + 1) <= a, k + 1, k)
        p = torch.where(a > 1.75 * torch.exp2(k), k - 7, k - 8).clamp(min=-117)  # scale 2^p
        u = (blk / torch.exp2(p)).abs()
        ku = torch.floor(torch.log2(u.clamp(min=2.0 ** -6)))
        ku = torch.where(torch.exp2(ku + 1) <= u, ku + 1, ku)
        step = torch.exp2(ku.clamp(min=-6) - 3)                                  # three fraction bits
        out[:, b:b + 128] = torch.sign(blk) * torch.round(u / step) * step * torch.exp2(p)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "lookup":
        v, d, ids = s["v"], s["d"], s["ids"]
        out = torch.zeros(s["t"], d, dtype=torch.float64, device=DEV)
        at = torch.nonzero((ids >= 0) & (ids < v)).view(-1)
        out[at] = s["params"][:v * d].view(v, d)[ids[at]].double() * s["scale"]
        return out
    if op == "emb_grad":
        v, d, ids = s["v"], s["d"], s["ids"]
        full = s["acc"].double()
        a = full[:v * d].view(v, d)
        at = torch.nonzero((ids >= 0) & (ids < v)).view(-1)
        a.index_add_(0, ids[at], s["dy"][at].double() * s["scale"])
        if s["emit"]:
            full[v * d:] = 0
        return full
    if op == "norm":
        h = (s["x"].double() + s["res"].double()).to(torch.bfloat16)   # h is held in bf16 by definition
        rstd = (h.double().square().mean(1) + EPS) ** -0.5
        y = _exact_act8(h.double() * rstd.unsqueeze(1) * s["params"][:s["d"]].double())
        return {"h": h.double(), "rstd": rstd, "y": y}
    if op == "norm_grad":
        d = s["d"]
        w, h, r, dy = s["params"][:d].double(), s["h"].double(), s["rstd"].double().unsqueeze(1), s["dy"].double()
        n = h * r                                                      # the normed row; y = n w
        dn = dy * w
        dx = s["dh"].double() + (dn - n * (dn * n).sum(1, keepdim=True) / d) * r
        acc = s["acc"].double()
        acc[:d] += s["scale"] * (dy * n).sum(0)
        return {"dx": dx, "acc": acc}
    if op == "act8":
        return _exact_act8(s["x"].double())
    o, i = s["o"], s["i"]
    scale = torch.exp2(s["e"].double() - 127).repeat_interleave(128, 1)[:, :i]
    x, dy = s["q"].double() * scale, s["dy"].double()
    acc = s["acc"].double()
    for b in range(0, i, 1024):
        xb = x[:, b:b + 1024].contiguous()
        if s["tr"]:
            acc[:o * i].view(i, o)[b:b + 1024] += s["scale"] * (xb.t().contiguous() @ dy)
        else:
            acc[:o * i].view(o, i)[:, b:b + 1024] += s["scale"] * (dy.t().contiguous() @ xb)
    return acc
