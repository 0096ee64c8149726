"""The gated linear recurrence and the RMS norm: what is measured of them.

Each case is one call that a program makes of ``wkv_recurrence_b200`` (or, for
training, the forward with its backward). Where ``own`` is false, ``run``
computes the same from elementary torch operations.

The recurrence, per channel of [B, T, C] inputs x and z with a carried state h:

    h_t = f_t h_{t-1} + i_t x_t      gate "sigmoid": f = sigmoid(z), i = 1 - f
                                     gate "decay":   f = e^{-z},     i = 1

The norm, over each of ``groups`` equal parts (heads) of a row of C columns:

    s = x + residual (held in the residual's type),
    y = s / sqrt(mean(s^2) + eps) * weight,

given in 16 or 32 bits, or in e4m3 with a scale per row or per block of columns.
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of a few interactive streams: latency is all there is
        dict(name="step 16 x 768 f32", op="step", B=16, C=768, x="f32", z="f32", gate="sigmoid"),
        # the decode workload of the benchmark: 4096 streams take a token each
        dict(name="step 4096 x 768 bf16", op="step", B=4096, C=768, x="bf16", z="bf16", gate="sigmoid"),
        # one very long document, slow and fast decays side by side
        dict(name="forward 1 x 65536 x 2048 f32", op="forward", B=1, T=65536, C=2048, x="f32", z="f32", out="f32",
             gate="decay", halves=False, starts=False),
        # rows packed from several documents (a gate of -inf starts each), x and z the two halves of one
        # projection, odd sizes
        dict(name="forward 3 x 1801 x 515 bf16 packed", op="forward", B=3, T=1801, C=515, x="bf16", z="bf16", out="bf16",
             gate="sigmoid", halves=True, starts=True),
        # a training step of one layer at the benchmark's layer shape
        dict(name="train 8 x 1024 x 768 bf16", op="train", B=8, T=1024, C=768, x="bf16", z="bf16", out="bf16",
             gate="sigmoid", halves=False, starts=False),
        # a training step of a wide layer: the benchmark's mixed shape, the decays held in 32 bits
        dict(name="train 16 x 4096 x 4096 bf16", op="train", B=16, T=4096, C=4096, x="bf16", z="f32", out="bf16",
             gate="decay", halves=False, starts=False),
        # the norm before a decode step's projections
        dict(name="norm 64 x 768 bf16", op="norm", N=64, C=768, groups=1, x="bf16", res="bf16", y="bf16"),
        # the norm of a prefill chunk over a residual stream held in 32 bits
        dict(name="norm 8192 x 4096 bf16 res f32", op="norm", N=8192, C=4096, groups=1, x="bf16", res="f32", y="bf16"),
        # a few streams' activations for 8-bit products, one scale a row
        dict(name="quant 16 x 4096 bf16", op="quant", N=16, C=4096, groups=1, x="bf16", res="bf16", block=0),
        # a large prefill's activations for 8-bit products, one scale for each 128 columns
        dict(name="quant 65536 x 4096 bf16 block 128", op="quant", N=65536, C=4096, groups=1, x="bf16", res="bf16",
             block=128),
        # the per-head norm of a readout (12 heads x 64), its gradients, an odd number of rows
        dict(name="norm backward 8191 x 12 x 64 f32", op="norm_backward", N=8191, C=768, groups=12, y="f32", s="f32",
             gs=False),
        # the gradients of a training step's norm, with the residual branch's own gradient
        dict(name="norm backward 65536 x 2048 bf16", op="norm_backward", N=65536, C=2048, groups=1, y="bf16", s="bf16",
             gs=True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["step", "forward", "train", "norm", "quant", "norm_backward"])
    if op in ("step", "forward", "train"):
        x = rng.choice(["f32", "bf16"])
        z = rng.choice(["f32", x])
        gate = rng.choice(["sigmoid", "decay"])
        C = _log(rng, 16, 4200)
        C = C if rng.random() < 0.4 else -(-C // 64) * 64
        if op == "step":
            return dict(op=op, B=_log(rng, 1, 8192), C=C, x=x, z=z, gate=gate)
        T = _log(rng, 1, 65536)
        B = max(1, min(_log(rng, 1, 64), (1 << 27) // (T * C)))
        T = min(T, (1 << 27) // (B * C))
        return dict(op=op, B=B, T=T, C=C, x=x, z=z, out=rng.choice(["f32", x]), gate=gate,
                    halves=x == z and rng.random() < 0.4, starts=gate == "sigmoid" and rng.random() < 0.3)
    D = rng.choice([32, 64, 96, 128, 256])
    groups = rng.choice([1, 1, 4, 12])
    C = D * groups if groups > 1 else _log(rng, 32, 16384)
    C = C if groups > 1 or rng.random() < 0.3 else -(-C // 128) * 128
    N = min(_log(rng, 1, 65536), (1 << 27) // C)
    x = rng.choice(["f32", "bf16"])
    if op == "norm_backward":
        return dict(op=op, N=N, C=C, groups=groups, y=x, s=rng.choice(["f32", x]), gs=rng.random() < 0.6)
    res = rng.choice(["none", "f32", x])
    if op == "norm":
        return dict(op=op, N=N, C=C, groups=groups, x=x, res=res, y=x)
    return dict(op=op, N=N, C=C, groups=groups, x=x, res=res, block=rng.choice([0, 128]) if C % 128 == 0 else 0)


# ----------------------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, dtype, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda").mul_(scale).to(dtype)

    def uniform(shape):
        return torch.rand(shape, generator=gen, device="cuda")

    op, C = case["op"], case["C"]
    st = dict(case)
    if op in ("step", "forward", "train"):
        xt, zt = _TYPES[case["x"]], _TYPES[case["z"]]
        B = case["B"]
        shape = (B, C) if op == "step" else (B, case["T"], C)
        if case.get("halves"):
            both = torch.empty(shape[:-1] + (2 * C,), dtype=xt, device="cuda")
            x, z = both[..., :C], both[..., C:]
        else:
            x, z = torch.empty(shape, dtype=xt, device="cuda"), torch.empty(shape, dtype=zt, device="cuda")
        x.copy_(normal(shape, torch.float32))
        if case["gate"] == "sigmoid":  # a gate that remembers tens of tokens, some channels thousands
            z.copy_(normal(shape, torch.float32, 1.5) + 1.0 + 7.0 * uniform((C,)))
        else:                          # decays log-uniform over [1e-4, 4]
            z.copy_(torch.exp(math.log(1e-4) + (math.log(4.0) - math.log(1e-4)) * uniform(shape)))
        if case.get("starts"):         # a document starts at about one token in 200
            z.masked_fill_((uniform(shape[:2]) < 0.005)[..., None], -math.inf)
        st.update(x=x, z=z, state=normal((B, C), torch.float32))
        if op == "train":
            st.update(g=normal(shape, _TYPES[case["out"]]), dstate=normal((B, C), torch.float32))
        return st
    N = case["N"]
    st["weight"] = 1.0 + normal((C,), torch.float32, 0.2)
    if op == "norm_backward":
        st["gy"] = normal((N, C), _TYPES[case["y"]])
        st["s"] = normal((N, C), _TYPES[case["s"]], 3.0)
        st["gs"] = normal((N, C), _TYPES[case["s"]]) if case["gs"] else None
    else:
        st["x"] = normal((N, C), _TYPES[case["x"]])
        st["residual"] = None if case["res"] == "none" else normal((N, C), _TYPES[case["res"]], 3.0)
    return st


# ----------------------------------------------------------------------------- the framework's calls

def _run_own(st):
    import wkv_recurrence_b200 as wkv

    op = st["op"]
    if op == "step":
        return wkv.gated_step(st["state"], st["x"], st["z"], gate=st["gate"])
    if op == "forward":
        return wkv.gated_forward(st["x"], st["z"], st["state"], gate=st["gate"], out_dtype=_TYPES[st["out"]])
    if op == "train":
        x, z, h0 = st["x"], st["z"], st["state"]
        marks = wkv.gated_checkpoints(x)
        out, state = wkv.gated_forward(x, z, h0, gate=st["gate"], out_dtype=_TYPES[st["out"]], checkpoints=marks)
        dx, dz, dh0 = wkv.gated_backward(x, z, st["g"], h0, st["dstate"], gate=st["gate"], checkpoints=marks)
        return out, state, dx, dz, dh0
    if op == "norm":
        return wkv.rms_norm(st["x"], st["weight"], st["residual"], eps=EPS, groups=st["groups"])
    if op == "quant":
        return wkv.rms_norm_quant(st["x"], st["weight"], st["residual"], eps=EPS, groups=st["groups"],
                                  block=st["block"])
    return wkv.rms_norm_backward(st["gy"], st["s"], st["weight"], st["gs"], eps=EPS, groups=st["groups"])


# ----------------------------------------------------------------------------- the plain form

def _coefficients(z, gate):
    """f and i of every token. In 64 bits: beside a gate near 1, what 1 - f loses in 32 bits adds up over the
    thousands of tokens that the channel remembers."""
    z = z.double()
    if gate == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-z)), 1.0 / (1.0 + torch.exp(z))
    return torch.exp(-z), torch.ones_like(z)


def _scan(f, b):
    """h_t = f_t h_{t-1} + b_t for t = 0.. (h before them 0) along dim 1, by doubling: after the pass with
    distance n, (f, b) of a token stand for the 2n tokens that end there. Overwrites f and b."""
    n = 1
    while n < f.shape[1]:
        b[:, n:] += f[:, n:] * b[:, :-n]
        f[:, n:] = f[:, n:] * f[:, :-n]
        n *= 2
    return b


def _recurrence(x, z, h0, gate):
    f, i = _coefficients(z, gate)
    b = i.mul_(x)
    b[:, 0] += f[:, 0] * h0
    return _scan(f, b)


def _gradients(x, z, h0, g, dstate, h, gate):
    f, i = _coefficients(z, gate)
    d = g.double()
    d[:, -1] += dstate
    after = torch.zeros_like(f)                   # f of the next token
    after[:, :-1] = f[:, 1:]
    d = _scan(after.flip(1), d.flip(1)).flip(1)   # dL/dh_t, all later tokens included
    del after
    before = torch.empty_like(h)                  # h of the token before
    before[:, 0] = h0
    before[:, 1:] = h[:, :-1]
    dh0 = f[:, 0] * d[:, 0]
    if gate == "sigmoid":
        dz = before.sub_(x).mul_(d).mul_(f).mul_(i)
    else:
        dz = before.mul_(d).mul_(f).neg_()
    return d.mul_(i), dz, dh0


def _sum(st):
    x, res = st["x"], st["residual"]
    return x if res is None else (x.float() + res.float()).to(res.dtype)


def _unit(s, groups):
    """s over the root of its mean square, by group, and that root's inverse."""
    s = s.float().view(s.shape[0], groups, -1)
    r = 1.0 / torch.sqrt((s * s).mean(-1, keepdim=True) + EPS)
    return s * r, r


def _run_plain(st):
    op = st["op"]
    if op == "step":
        f, i = _coefficients(st["z"], st["gate"])
        h = f * st["state"] + i * st["x"]
        return h.to(st["x"].dtype), h.float()
    if op in ("forward", "train"):
        x, z, h0, gate = st["x"], st["z"], st["state"], st["gate"]
        h = _recurrence(x, z, h0, gate)
        out, state = h.to(_TYPES[st["out"]]), h[:, -1].float()
        if op == "forward":
            return out, state
        dx, dz, dh0 = _gradients(x, z, h0, st["g"], st["dstate"], h, gate)
        return out, state, dx.to(x.dtype), dz.to(z.dtype), dh0.float()
    groups, w = st["groups"], st["weight"]
    if op == "norm_backward":
        unit, r = _unit(st["s"], groups)
        gy = st["gy"].float().view_as(unit)
        p = gy * w.view(1, groups, -1)
        ds = ((p - unit * (p * unit).mean(-1, keepdim=True)) * r).view(st["s"].shape)
        dw = (gy * unit).double().sum(0).float().view(-1)  # a long sum over the rows
        if st["gs"] is not None:
            ds = ds + st["gs"].float()
        return ds.to(st["s"].dtype), dw
    s = _sum(st)
    y = (_unit(s, groups)[0] * w.view(1, groups, -1)).view(s.shape)
    s = None if st["residual"] is None else s
    if op == "norm":
        return y.to(st["x"].dtype), s
    block = st["block"] or y.shape[1]
    parts = y.view(y.shape[0], -1, block)
    top = parts.abs().amax(-1, keepdim=True)
    scale = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    q = (parts / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(y.shape)
    return q, scale.squeeze(-1), s


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("step", "forward", "train"):
        x, z = st["x"], st["z"]
        h = st["state"].double()
        if op == "step":
            x, z = x[:, None], z[:, None]
        T = x.shape[1]

        def gate(t):
            zt = z[:, t].double()
            if case["gate"] == "sigmoid":
                return torch.sigmoid(zt), torch.sigmoid(-zt)
            return torch.exp(-zt), torch.ones_like(zt)

        hs = [h]
        for t in range(T):
            f, i = gate(t)
            h = f * h + i * x[:, t].double()
            hs.append(h)
        if op == "step":
            return h, h
        if op == "forward":
            return torch.stack(hs[1:], 1), h
        dx, dz = [None] * T, [None] * T
        q = st["dstate"].double()
        for t in range(T - 1, -1, -1):
            f, i = gate(t)
            d = st["g"][:, t].double() + q
            dx[t] = i * d
            dz[t] = d * (hs[t] - x[:, t].double()) * f * i if case["gate"] == "sigmoid" else -d * hs[t] * f
            q = f * d
        return torch.stack(hs[1:], 1), h, torch.stack(dx, 1), torch.stack(dz, 1), q
    G, C, N = case["groups"], case["C"], case["N"]
    D = C // G
    w = st["weight"].double().view(G, D)
    if op == "norm_backward":
        s, gy = st["s"].double().view(N, G, D), st["gy"].double().view(N, G, D)
        var = s.pow(2).sum(-1) / D + EPS
        dot = (gy * w * s).sum(-1)
        ds = gy * w * var.rsqrt()[..., None] - s * (dot / (D * var * var.sqrt()))[..., None]
        if st["gs"] is not None:
            ds = ds + st["gs"].double().view(N, G, D)
        dw = torch.einsum("ngd,ngd,ng->gd", gy, s, var.rsqrt())
        return ds.view(N, C), dw.reshape(C)
    s = st["x"].double()
    if st["residual"] is not None:
        s = (s + st["residual"].double()).to(st["residual"].dtype).double()
    heads = s.view(N, G, D)
    y = (heads * w / (heads.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt()).view(N, C)
    held = None if st["residual"] is None else s
    if op == "norm":
        return y, held
    block = case["block"] or C
    scale = y.view(N, C // block, block).abs().amax(-1) / E4M3_MAX
    scale = scale.masked_fill(scale == 0, 1.0)
    return (y.view(N, C // block, block) / scale[..., None]).view(N, C), scale, held


# ----------------------------------------------------------------------------- work

def work(case):
    size = {"f32": 4, "bf16": 2, "none": 0}
    op, C = case["op"], case["C"]
    if op in ("step", "forward", "train"):
        n = case["B"] * case.get("T", 1) * C
        x, z = size[case["x"]], size[case["z"]]
        out = size[case["out"]] if op != "step" else x
        state = 4 * case["B"] * C
        if op == "train":  # x, z, g in; out, dx, dz out; four states
            return {"bytes": n * (2 * x + 2 * z + 2 * out) + 4 * state, "flops": 20 * n}
        return {"bytes": n * (x + z + out) + 2 * state, "flops": 8 * n}
    n = case["N"] * C
    if op == "norm_backward":
        s = size[case["s"]]
        return {"bytes": n * (size[case["y"]] + s * (3 if case["gs"] else 2)) + 8 * C, "flops": 12 * n}
    res = size[case["res"]]
    bytes_in = n * (size[case["x"]] + 2 * res) + 4 * C
    if op == "norm":
        return {"bytes": bytes_in + n * size[case["y"]], "flops": 5 * n}
    return {"bytes": bytes_in + n + 4 * case["N"] * (C // (case["block"] or C)), "flops": 8 * n}
