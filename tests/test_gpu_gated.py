"""The gated linear recurrence on the GPU against its float64 oracle: forward,
backward and step over types, gates, lengths around every tile edge, odd
widths, strides, sequence starts, and the ways a program calls them."""
import numpy as np
import pytest
import torch

import wkv_recurrence_b200 as W
from oracle import gated_oracle as G

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TYPES = [(F32, F32, F32), (BF16, BF16, BF16), (BF16, BF16, F32), (BF16, F32, BF16), (BF16, F32, F32)]
# half a step of the output's type, relative to the value
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


def draw(B, T, C, xt, zt, gate, seed=0, starts=False, slow=False):
    g = torch.Generator(device="cuda").manual_seed(1000 * T + C + seed)
    x = torch.randn(B, T, C, generator=g, device="cuda").to(xt)
    if gate == "sigmoid":
        z = torch.randn(B, T, C, generator=g, device="cuda") * 2 + (8 if slow else 1)
    else:
        z = torch.exp(torch.rand(B, T, C, generator=g, device="cuda") * (2 if slow else 10.6) - 9.2)
    z = z.to(zt)
    if starts and T > 0:
        at = torch.rand(B, T, generator=g, device="cuda") < 0.05
        z[at] = -np.inf if gate == "sigmoid" else np.inf
    h0 = torch.randn(B, C, generator=g, device="cuda")
    return x, z, h0


def np64(t):
    return t.detach().double().cpu().numpy()


def check(got, ref, allowed, what):
    half = HALF[got.dtype]
    got = np64(got)
    assert got.shape == ref.shape, what
    lim = (np.abs(ref) + allowed) * half + allowed + 1e-37  # underflow: results below the smallest normal are flushed
    bad = ~(np.abs(got - ref) <= lim)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:3], ref[bad][:3], lim[bad][:3])


def check_forward(x, z, h0, gate, out, state):
    ref, rst = G.forward(np64(x), np64(z), None if h0 is None else np64(h0), gate)
    al, _ = G.allowed_forward(np64(x), np64(z), None if h0 is None else np64(h0), gate)
    check(out, ref, al, "out")
    if x.shape[1]:
        check(state, rst, al[:, -1], "state")


def check_backward(x, z, h0, g, ds, gate, got):
    args = (np64(x), np64(z), None if h0 is None else np64(h0), np64(g), None if ds is None else np64(ds), gate)
    for a, r, al, what in zip(got, G.backward(*args), G.allowed_backward(*args), ("dx", "dz", "dstate")):
        check(a, r, al, what)


@pytest.mark.parametrize("gate", ["sigmoid", "decay"])
@pytest.mark.parametrize("xt,zt,ot", TYPES)
@pytest.mark.parametrize("B,T,C", [(2, 1, 64), (1, 17, 3), (2, 128, 66), (3, 129, 65), (2, 517, 130)])
def test_forward_and_backward(B, T, C, xt, zt, ot, gate):
    x, z, h0 = draw(B, T, C, xt, zt, gate)
    marks = W.gated_checkpoints(x)
    out, state = W.gated_forward(x, z, h0, gate=gate, out_dtype=ot, checkpoints=marks)
    assert out.dtype == ot
    check_forward(x, z, h0, gate, out, state)
    g = torch.randn(B, T, C, device="cuda").to(ot)
    ds = torch.randn(B, C, device="cuda")
    got = W.gated_backward(x, z, g, h0, ds, gate=gate, checkpoints=marks)
    assert got[0].dtype == xt and got[1].dtype == zt
    check_backward(x, z, h0, g, ds, gate, got)
    again = W.gated_backward(x, z, g, h0, ds, gate=gate)  # without the forward's checkpoints
    for a, b in zip(got, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 112, 127, 128, 129, 143, 144, 145, 255, 256, 257, 2047, 2048,
                               2049, 4113])
@pytest.mark.parametrize("C", [1, 2, 33, 64])
def test_lengths_and_widths(T, C):
    x, z, h0 = draw(2, T, C, F32, F32, "sigmoid", seed=1)
    out, state = W.gated_forward(x, z, h0)
    check_forward(x, z, h0, "sigmoid", out, state)
    g, ds = torch.randn_like(x), torch.randn_like(h0)
    check_backward(x, z, h0, g, ds, "sigmoid", W.gated_backward(x, z, g, h0, ds))


@pytest.mark.parametrize("gate", ["sigmoid", "decay"])
@pytest.mark.parametrize("T", [5, 200, 3000])
def test_sequence_starts_and_no_state(T, gate):
    x, z, _ = draw(2, T, 40, F32, F32, gate, seed=2, starts=True)
    z[0, 0] = -np.inf if gate == "sigmoid" else np.inf
    z[1, T - 1] = -np.inf if gate == "sigmoid" else np.inf
    out, state = W.gated_forward(x, z, gate=gate)
    check_forward(x, z, None, gate, out, state)
    g = torch.randn_like(x)
    dx, dz, dh = W.gated_backward(x, z, g, gate=gate)
    check_backward(x, z, None, g, None, gate, (dx, dz, dh))
    assert torch.equal(dz[z.isinf()], torch.zeros_like(dz[z.isinf()]))  # nothing flows through a start
    assert torch.equal(out[1, T - 1], x[1, T - 1])


def test_a_held_state_passes_a_gate_of_infinity_exactly():
    x, z, h0 = draw(1, 300, 64, F32, F32, "sigmoid")
    z.fill_(np.inf)
    out, state = W.gated_forward(x, z, h0)
    assert torch.equal(out, h0[:, None].expand_as(out)) and torch.equal(state, h0)
    zd = torch.zeros_like(x)
    zd[:, ::2] = -0.0
    out, state = W.gated_forward(torch.zeros_like(x), zd, h0, gate="decay")
    assert torch.equal(out, h0[:, None].expand_as(out)) and torch.equal(state, h0)


def test_constant_slow_gate_keeps_its_mean():
    """1 - f = 1e-4 for 40000 tokens of a constant input, in closed form."""
    T = 40000
    x = torch.ones(1, T, 34, device="cuda")
    z = torch.full((1, T, 34), 9.0, device="cuda") + torch.arange(34, device="cuda") * 0.01
    out, state = W.gated_forward(x, z)
    check_forward(x, z, None, "sigmoid", out, state)
    # a constant input approaches it as 1 - (1 - m)^T: at z = 9.33, m = 8.9e-5, that is 1 - e^{-3.55} = 0.971
    m = 1 / (1 + np.exp(np64(z)[0, 0]))
    want = -np.expm1(T * np.log1p(-m))
    # the state stays below 1 and is rounded by at most 2^-25 twice a token; 1/m = 1.1e4 tokens of such errors are
    # remembered: 6.7e-4. The gate's own error, (9.33 + 8) 2^-23 of m, moves 1 - e^{-Tm} by less than 1e-6.
    assert np.abs(np64(out)[0, -1] - want).max() < 7e-4
    zd = torch.full((1, T, 34), 1e-4, device="cuda")
    out, state = W.gated_forward(x, zd, gate="decay")
    ref, _ = G.forward(np64(x), np64(zd), None, "decay")
    # the sum's fixed point is 1 / (1 - f) = 1e4; the recurrence forgets errors over as many tokens
    assert np.abs(np64(out) / ref - 1).max() < 1e4 * 2 * 2.0 ** -23


@pytest.mark.parametrize("T", [60, 300])
def test_growing_decay(T):
    x, z, h0 = draw(1, T, 8, F32, F32, "decay")
    z = -0.05 * torch.rand_like(z)  # f > 1
    out, state = W.gated_forward(x, z, h0, gate="decay")
    check_forward(x, z, h0, "decay", out, state)


@pytest.mark.parametrize("B,T,C", [(20, 300, 2048), (600, 140, 30), (1, 40000, 40)])
def test_many_groups_and_long_rows(B, T, C):
    x, z, h0 = draw(B, T, C, F32, F32, "sigmoid", slow=True)
    marks = W.gated_checkpoints(x)
    out, state = W.gated_forward(x, z, h0, checkpoints=marks)
    g, ds = torch.randn_like(x), torch.randn_like(h0)
    got = W.gated_backward(x, z, g, h0, ds, checkpoints=marks)
    rows = slice(0, 2) if B > 2 else slice(0, 1)
    cols = slice(0, min(C, 70))
    cut = lambda t: t[rows][..., cols].contiguous()  # noqa: E731
    check_forward(cut(x), cut(z), cut(h0), "sigmoid", cut(out), cut(state))
    check_backward(cut(x), cut(z), cut(h0), cut(g), cut(ds), "sigmoid", [cut(t) for t in got])
    last = slice(B - 1, B)
    tail = slice(max(0, C - 33), C)
    cut = lambda t: t[last][..., tail].contiguous()  # noqa: E731
    check_forward(cut(x), cut(z), cut(h0), "sigmoid", cut(out), cut(state))
    check_backward(cut(x), cut(z), cut(h0), cut(g), cut(ds), "sigmoid", [cut(t) for t in got])
    out2, state2 = W.gated_forward(x, z, h0)
    assert torch.equal(out, out2) and torch.equal(state, state2)  # bitwise reproducible
    for a, b in zip(got, W.gated_backward(x, z, g, h0, ds, checkpoints=marks)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [100, 400])
def test_strides_and_alignment(T):
    B, C = 3, 66
    both = torch.randn(B, T, 2 * C + 1, device="cuda").to(BF16)
    for x, z in ((both[..., :C], both[..., C:2 * C]),              # halves of one projection, odd row pitch
                 (both[..., 1:C + 1], both[..., C + 1:2 * C + 1]),  # a base that only fits one element
                 (both.transpose(0, 1).contiguous().transpose(0, 1)[..., :C], both[..., C:2 * C]),  # time first
                 (both[..., :C], both[:1, :, C:2 * C].expand(B, T, C)),  # one gate for all rows
                 (both[..., :C], both[:, :1, C:2 * C].expand(B, T, C))):  # one gate for all tokens
        out, state = W.gated_forward(x, z)
        want, wst = W.gated_forward(x.contiguous(), z.contiguous())
        check_forward(x, z, None, "sigmoid", out, state)
        g = torch.randn(B, T, C, device="cuda").to(BF16)
        check_backward(x, z, None, g, None, "sigmoid", W.gated_backward(x, z, g))
        assert torch.equal(out, want) and torch.equal(state, wst)


def test_time_of_zero_and_empty_batches():
    h0 = torch.randn(2, 5, device="cuda")
    e = torch.empty(2, 0, 5, device="cuda")
    out, state = W.gated_forward(e, e, h0)
    assert out.shape == (2, 0, 5) and torch.equal(state, h0)
    assert torch.equal(W.gated_forward(e, e)[1], torch.zeros_like(h0))
    dx, dz, dh = W.gated_backward(e, e, e, h0, h0)
    assert dx.numel() == 0 and torch.equal(dh, h0)
    for shape in ((0, 7, 5), (2, 7, 0)):
        e = torch.empty(shape, device="cuda")
        assert W.gated_forward(e, e)[0].shape == shape
        assert W.gated_backward(e, e, e)[0].shape == shape
    s = torch.empty(0, 4, device="cuda")
    assert W.gated_step(s, s, s)[0].shape == (0, 4)


@pytest.mark.parametrize("T", [20, 100, 300, 5000])
def test_state_in_place_and_split(T):
    x, z, h0 = draw(2, T, 96, F32, F32, "sigmoid")
    out, state = W.gated_forward(x, z, h0)
    s = h0.clone()
    o2, s2 = W.gated_forward(x, z, s, state_out=s)
    assert s2 is s and torch.equal(o2, out) and torch.equal(s, state)
    k = T // 3  # hand the state over in the middle
    a, s = W.gated_forward(x[:, :k], z[:, :k], h0)
    b, s = W.gated_forward(x[:, k:], z[:, k:], s)
    check_forward(x, z, h0, "sigmoid", torch.cat([a, b], 1), s)


@pytest.mark.parametrize("gate", ["sigmoid", "decay"])
@pytest.mark.parametrize("xt,zt,ot", TYPES)
@pytest.mark.parametrize("S,C", [(1, 1), (5, 66), (64, 768), (3, 4100)])
def test_step(S, C, xt, zt, ot, gate):
    x, z, h0 = draw(S, 1, C, xt, zt, gate)
    out, state = W.gated_step(h0, x[:, 0], z[:, 0], gate=gate, out_dtype=ot)
    check_forward(x, z, h0, gate, out[:, None], state)
    wide = torch.zeros(S, 2 * C + 1, device="cuda", dtype=xt)
    wide[:, :C] = x[:, 0]
    s = h0.clone()
    o2, s2 = W.gated_step(s, wide[:, :C], z[:, 0], gate=gate, out_dtype=ot, inplace=True)
    assert s2 is s and torch.equal(s, state) and torch.equal(o2, out)


def test_steps_follow_the_sequence():
    x, z, h0 = draw(3, 40, 64, F32, F32, "decay")
    out, state = W.gated_forward(x, z, h0, gate="decay")
    s = h0.clone()
    for t in range(40):
        o, s = W.gated_step(s, x[:, t], z[:, t], gate="decay", inplace=True)
        al, _ = G.allowed_forward(np64(x), np64(z), np64(h0), "decay")
        assert (np.abs(np64(o) - np64(out[:, t])) <= 2 * al[:, t] + 1e-6 * np.abs(np64(o))).all()


def test_autograd_and_differences():
    for gate in ("sigmoid", "decay"):
        x, z, h0 = draw(2, 150, 4, F32, F32, gate, seed=9)
        x, z, h0 = (t.requires_grad_() for t in (x, z, h0))
        out, state = W.Gated.apply(x, z, h0, gate)
        g, ds = torch.randn_like(out), torch.randn_like(state)
        dx, dz, dh = torch.autograd.grad((out * g).sum() + (state * ds).sum(), (x, z, h0))
        check_backward(x, z, h0, g, ds, gate, (dx, dz, dh))
        # and against differences of the float64 forward: the central difference of step d is off by d^2/6 times a
        # third derivative of order |gradient|, and by 2^-52 |loss| / d
        args = [np64(t) for t in (x, z, h0)]
        loss = lambda a: float((G.forward(*a, gate)[0] * np64(g)).sum() + (G.forward(*a, gate)[1] * np64(ds)).sum())  # noqa: E731
        rng = np.random.default_rng(1)
        for k, grad in enumerate((dx, dz, dh)):
            for _ in range(4):
                at = tuple(rng.integers(0, n) for n in args[k].shape)
                d = 1e-4 * (1.0 if k != 1 or gate == "sigmoid" else max(1e-1, args[1][at]))
                up, down = [a.copy() for a in args], [a.copy() for a in args]
                up[k][at] += d
                down[k][at] -= d
                want = (loss(up) - loss(down)) / (2 * d)
                assert abs(float(grad[at]) - want) <= 1e-4 * max(1.0, abs(want)), (gate, k, at)
    # a shared gate's gradient is summed over what shares it; outputs that are not used give zeros
    x, z, _ = draw(3, 140, 8, BF16, BF16, "sigmoid")
    zs = z[:1].clone().requires_grad_()
    out, _ = W.Gated.apply(x, zs.expand(3, 140, 8), None, "sigmoid")
    out.float().sum().backward()
    want = G.backward(np64(x), np64(z[:1].expand(3, 140, 8)), None, np.ones(x.shape), None, "sigmoid")[1].sum(0, keepdims=True)
    al = G.allowed_backward(np64(x), np64(z[:1].expand(3, 140, 8)), None, np.ones(x.shape), None, "sigmoid")[1].sum(0, keepdims=True)
    # three bf16 gradients, rounded once each and summed with two more bf16 roundings
    mag = np.abs(G.backward(np64(x), np64(z[:1].expand(3, 140, 8)), None, np.ones(x.shape), None, "sigmoid")[1]).sum(0, keepdims=True)
    assert (np.abs(np64(zs.grad) - want) <= 4 * 2.0 ** -8 * mag + al).all()
    xr = x.clone().requires_grad_()
    _, st = W.Gated.apply(xr, z, None, "sigmoid")
    st.sum().backward()
    check_backward(x, z, None, torch.zeros_like(x), torch.ones(3, 8, device="cuda"), "sigmoid",
                   (xr.grad, *W.gated_backward(x, z, torch.zeros_like(x), None, torch.ones(3, 8, device="cuda"))[1:]))


def test_one_workspace_over_shapes_and_directions():
    ws = torch.zeros(W.gated_workspace_size(4, 3000, 200), dtype=torch.uint8, device="cuda")
    for (B, T, C) in ((4, 3000, 200), (1, 700, 64), (2, 2500, 199), (4, 3000, 200)):
        x, z, h0 = draw(B, T, C, F32, F32, "sigmoid")
        marks = W.gated_checkpoints(x)
        out, state = W.gated_forward(x, z, h0, workspace=ws, checkpoints=marks)
        g = torch.randn_like(x)
        got = W.gated_backward(x, z, g, h0, workspace=ws, checkpoints=marks)
        assert W.query_status(ws) == 0
        check_forward(x[:1], z[:1], h0[:1], "sigmoid", out[:1], state[:1])
        check_backward(x[:1], z[:1], h0[:1], g[:1], None, "sigmoid", [t[:1] for t in got])


def test_two_streams_at_once():
    jobs = []
    for i in range(2):
        x, z, h0 = draw(2, 6000, 128, F32, F32, "sigmoid", seed=i)
        jobs.append((x, z, h0, W.gated_forward(x, z, h0)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[] for _ in jobs]
    for _ in range(5):
        for i, (x, z, h0, _) in enumerate(jobs):
            with torch.cuda.stream(streams[i]):
                got[i].append(W.gated_forward(x, z, h0))
    torch.cuda.synchronize()
    for i, (_, _, _, want) in enumerate(jobs):
        for out, state in got[i]:
            assert torch.equal(out, want[0]) and torch.equal(state, want[1])


def test_graphs_captured_on_one_stream_and_replayed_on_two():
    jobs = []
    side = torch.cuda.Stream()
    for i in range(2):
        x, z, h0 = draw(2, 5000, 128, F32, F32, "sigmoid", seed=i)
        g = torch.randn_like(x)
        marks = W.gated_checkpoints(x)
        want = (*W.gated_forward(x, z, h0, checkpoints=marks), *W.gated_backward(x, z, g, h0, checkpoints=marks))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            m = W.gated_checkpoints(x)
            got = (*W.gated_forward(x, z, h0, checkpoints=m), *W.gated_backward(x, z, g, h0, checkpoints=m))
        jobs.append((graph, want, got, (x, z, h0, g)))
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(4):
        for s, (graph, *_) in zip(streams, jobs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, want, got, _ in jobs:
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    x = jobs[0][3][0]
    x.copy_(torch.randn_like(x))  # new inputs in the captured tensors
    jobs[0][0].replay()
    torch.cuda.synchronize()
    want = W.gated_forward(*jobs[0][3][:3])
    assert torch.equal(jobs[0][2][0], want[0]) and torch.equal(jobs[0][2][1], want[1])


def test_offsets_beyond_32_bits():
    """Rows whose token stride puts the last elements past 2^31 elements of the base."""
    T, C = 260, 64
    pitch = (1 << 31) // 250
    big = torch.empty(T * pitch, dtype=BF16, device="cuda")
    x = big.as_strided((1, T, C), (0, pitch, 1))
    z = torch.randn(1, T, C, device="cuda").to(BF16)
    x.copy_(torch.randn(1, T, C, device="cuda"))
    out, state = W.gated_forward(x, z)
    check_forward(x, z, None, "sigmoid", out, state)


DEBUG_CHILD = r'''
import numpy as np, torch, sys
sys.path.insert(0, "tests")
import wkv_recurrence_b200 as W
from wkv_recurrence_b200 import _abi
import test_gpu_gated as T
assert _abi.LIB_PATH.endswith("libwkv_debug.so"), _abi.LIB_PATH
checked = 0
for (B, L, C) in ((2, 517, 200), (3, 129, 65), (1, 65, 36), (300, 140, 70), (1, 5000, 33)):
    for xt, zt, ot in ((T.F32, T.F32, T.F32), (T.BF16, T.BF16, T.BF16), (T.BF16, T.F32, T.F32)):
        for gate in ("sigmoid", "decay"):
            x, z, h0 = T.draw(B, L, C, xt, zt, gate)
            ws = torch.zeros(W.gated_workspace_size(B, L, C), dtype=torch.uint8, device="cuda")
            marks = W.gated_checkpoints(x)
            out, st = W.gated_forward(x, z, h0, gate=gate, out_dtype=ot, checkpoints=marks, workspace=ws)
            g = torch.randn(B, L, C, device="cuda").to(ot)
            got = W.gated_backward(x, z, g, h0, gate=gate, checkpoints=marks, workspace=ws)
            assert W.query_status(ws) == 0, (B, L, C, xt, gate)
            k = slice(0, 2)
            T.check_forward(x[k], z[k], h0[k], gate, out[k], st[k])
            T.check_backward(x[k], z[k], h0[k], g[k], None, gate, [t[k] for t in got])
            checked += 1
print("checked", checked)
'''


def test_bounds_checked_build():
    import os
    import subprocess
    import sys

    from wkv_recurrence_b200 import build
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    build.build(debug=True)
    env = dict(os.environ, WKV_LIBRARY="debug", PYTHONPATH=root)
    r = subprocess.run([sys.executable, "-c", DEBUG_CHILD], cwd=root, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "checked 30" in r.stdout


def test_the_binding_refuses_on_the_gpu():
    x = torch.zeros(2, 200, 8, device="cuda")
    h = torch.zeros(2, 8, device="cuda")
    bad = [(lambda: W.gated_forward(x, x[:, :5]), ValueError), (lambda: W.gated_forward(x[0], x[0]), ValueError),
           (lambda: W.gated_forward(x.half(), x), TypeError), (lambda: W.gated_forward(x, x.bfloat16()), TypeError),
           (lambda: W.gated_forward(x.transpose(1, 2), x.transpose(1, 2)), ValueError),
           (lambda: W.gated_forward(x, x, gate="tanh"), ValueError), (lambda: W.gated_forward(x, x, gate=None), ValueError),
           (lambda: W.gated_forward(x, x, h[:1]), ValueError), (lambda: W.gated_forward(x, x, h.double()), TypeError),
           (lambda: W.gated_forward(x, x, h.cpu()), ValueError), (lambda: W.gated_forward(x, x, out_dtype=BF16), TypeError),
           (lambda: W.gated_forward(x, x, out_dtype="f32"), TypeError),
           (lambda: W.gated_forward(x, x, out=x[:, :, :4]), ValueError),
           (lambda: W.gated_forward(x, x, checkpoints=torch.zeros(2, 1, 8, device="cuda")), ValueError),
           (lambda: W.gated_forward(x, x, workspace=torch.zeros(300, dtype=torch.uint8)), ValueError),
           (lambda: W.gated_backward(x, x, x.bfloat16()), TypeError), (lambda: W.gated_backward(x, x, x[:, :3]), ValueError),
           (lambda: W.gated_backward(x, x, None), ValueError), (lambda: W.gated_step(h, x[:, 0], x[:, 0], out=h[:1]), ValueError),
           (lambda: W.gated_step(None, x[:, 0], x[:, 0]), ValueError),
           (lambda: W.gated_forward(x, x, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")), W.WkvError)]
    for call, kind in bad:
        with pytest.raises(kind):
            call()
    with pytest.raises(W.WkvError, match="wkv_gated_forward"):
        bad[-1][0]()


FIRST_CALL_CHILD = r'''
import torch, sys
import wkv_recurrence_b200 as W
x = torch.randn(2, 700, 96, device="cuda")
g, w = torch.randn_like(x), torch.ones(96, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    marks = W.gated_checkpoints(x)
    out, st = W.gated_forward(x, x, checkpoints=marks)
    got = W.gated_backward(x, x, g, checkpoints=marks)
    y, s = W.rms_norm(out, w, x)
    ds, dw = W.rms_norm_backward(g, s, w)
graph.replay()
torch.cuda.synchronize()
want, wst = W.gated_forward(x, x)
assert torch.equal(out, want) and torch.equal(st, wst)
assert all(torch.equal(a, b) for a, b in zip(got, W.gated_backward(x, x, g)))
y2, s2 = W.rms_norm(want, w, x)
d2, w2 = W.rms_norm_backward(g, s2, w)
assert torch.equal(y, y2) and torch.equal(ds, d2) and torch.equal(dw, w2)
print("the first call, captured")
'''


def test_the_first_call_of_a_process_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_CHILD], cwd=root, env=dict(os.environ, PYTHONPATH=root),
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "the first call, captured" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]


def test_a_wait_that_runs_out_is_reported():
    """A workspace whose records cannot come (the header says that all tickets are taken but the first tiles' records are
    missing) ends within the limit of each wait and says so."""
    B, T, C = 1, 260, 64  # three tiles; the calls below take tickets 1, 2 and 3 (past the end)
    ws = torch.zeros(W.gated_workspace_size(B, T, C), dtype=torch.uint8, device="cuda")
    ws[:4].view(torch.int32).fill_(1)  # the ticket of tile 0 is gone: its total never arrives
    x = torch.randn(B, T, C, device="cuda")
    W.gated_forward(x, x, workspace=ws)
    assert W.query_status(ws) == 6  # WKV_ERR_WAIT_TIMEOUT
    assert W.query_status(ws) == 0
    out, state = W.gated_forward(x, x, workspace=ws)  # the header is ready for the next call
    assert W.query_status(ws) == 0
    check_forward(x, x, None, "sigmoid", out, state)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_masks_of_the_types_extremes(dt):
    """finfo.min in a sigmoid gate (finfo.max in a decay) starts a sequence, the other end of a sigmoid gate keeps it:
    e^{+-3e38} is 0 or infinity in any precision."""
    for T in (40, 300):
        x, z, h0 = draw(2, T, 34, dt, dt, "sigmoid")
        z[:, T // 2] = torch.finfo(dt).min
        z[:, T // 3] = torch.finfo(dt).max
        out, state = W.gated_forward(x, z, h0)
        check_forward(x, z, h0, "sigmoid", out, state)
        assert torch.equal(out[:, T // 2], x[:, T // 2])
        g = torch.randn(2, T, 34, device="cuda").to(dt)
        check_backward(x, z, h0, g, None, "sigmoid", W.gated_backward(x, z, g, h0))
        xd, zd, h0 = draw(2, T, 34, dt, dt, "decay")
        zd[:, T // 2] = torch.finfo(dt).max
        zd[:, T // 3] = 0
        out, state = W.gated_forward(xd, zd, h0, gate="decay")
        check_forward(xd, zd, h0, "decay", out, state)
        assert torch.equal(out[:, T // 2], xd[:, T // 2])
        check_backward(xd, zd, h0, g, None, "decay", W.gated_backward(xd, zd, g, h0, gate="decay"))


def test_calls_from_two_host_threads():
    """Two threads, a stream each, at once: each has a workspace of its own."""
    import threading
    jobs = [draw(2, 3000, 128, F32, F32, "sigmoid", seed=i) for i in range(2)]
    want = [W.gated_forward(*j) for j in jobs]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    got[i].append(W.gated_forward(*jobs[i]))
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for i in range(2):
        for out, state in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(state, want[i][1])


def growth(kind, T, B, C):
    """Decays whose product is finite over a tile of 128 tokens (2^92 for z = -1/2) but not over several, on states that
    stay finite all the same."""
    g = torch.Generator(device="cuda").manual_seed(C + B)
    x, z = torch.zeros(B, T, C, device="cuda"), torch.zeros(B, T, C, device="cuda")
    h0 = torch.zeros(B, C, device="cuda")
    gr, ds = torch.zeros_like(x), torch.zeros_like(h0)
    noise = torch.randn(B, T, C, generator=g, device="cuda")
    if kind == "zero":  # nothing to grow up to the last token (the gradient: down to the first)
        z.fill_(-0.5)
        x[:, -1], gr[:, 0] = noise[:, -1], noise[:, 0]
    elif kind == "small":  # 1e-30 grows by 2^184 in two tiles
        z[:, 128 * 12:128 * 14] = -0.5
        h0, ds = 1e-30 * noise[:, 0], 1e-30 * noise[:, 1]
    elif kind == "start":  # growth of nothing, a start, and ordinary tokens behind it (in front of it for the gradient)
        z[:, :128 * 11] = -0.5
        z[:, 128 * 11] = np.inf
        x[:, 128 * 11:] = noise[:, 128 * 11:]
        z[:, 128 * 11 + 1:] = 0.01
        z[:, 128 * 25] = np.inf
        z[:, 128 * 25 + 1:] = -0.5
        x[:, 128 * 25:] = 0
        gr[:, 128 * 11:128 * 25] = noise[:, 128 * 11:128 * 25]
    else:  # two tiles up, two tiles down, again and again, up at either end
        z[:, :256 * 19] = torch.where(torch.arange(256 * 19, device="cuda") // 256 % 2 == 0, -0.5, 0.5)[None, :, None]
        h0, ds = 1e-30 * noise[:, 0], 1e-30 * noise[:, 1]
    return x, z, h0, gr, ds


@pytest.mark.parametrize("kind", ["zero", "small", "start", "waves"])
@pytest.mark.parametrize("B,C", [(1, 64), (50, 128), (300, 64)])  # look-back groups of 32 tiles, of 8 and of one
def test_growth_over_many_tiles(B, C, kind):
    x, z, h0, gr, ds = growth(kind, 128 * 40 + 17, B, C)
    marks = W.gated_checkpoints(x)
    out, state = W.gated_forward(x, z, h0, gate="decay", checkpoints=marks)
    got = W.gated_backward(x, z, gr, h0, ds, gate="decay", checkpoints=marks)
    for t in (out, state, *got):
        assert bool(t.isfinite().all())
    for row in {0, B - 1}:
        cut = lambda t: t[row:row + 1, ..., C - 9:].contiguous()  # noqa: E731
        check_forward(cut(x), cut(z), cut(h0), "decay", cut(out), cut(state))
        check_backward(cut(x), cut(z), cut(h0), cut(gr), cut(ds), "decay", [cut(t) for t in got])


def test_autograd_sees_what_was_written_in_place():
    """A backward whose saved tensor was overwritten raises, as behind torch's own in-place operators, instead of using
    what lies there now."""
    B, T, C = 2, 5, 16
    x, z, h0 = draw(B, T, C, F32, F32, "sigmoid")
    x.requires_grad_()
    other, marks = torch.randn_like(h0), W.gated_checkpoints(x)
    for overwrite in (lambda: W.gated_step(h0, x[:, 0], z[:, 0], inplace=True),
                      lambda: W.gated_step(other, x[:, 0], z[:, 0], state_out=h0),
                      lambda: W.gated_step(other, x[:, 0], z[:, 0], out=h0),
                      lambda: W.gated_forward(x, z, h0, state_out=h0),
                      lambda: W.gated_forward(x, z, h0, state_out=h0.view(1, B * C).view(B, C)),
                      lambda: W.gated_forward(x.detach(), z, out=z)):
        out, state = W.Gated.apply(x, z, h0, "sigmoid")
        overwrite()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            (out.sum() + state.sum()).backward()
    W.Gated.apply(x, z, h0, "sigmoid")[0].sum().backward()  # and nothing else counts as written
    v = [t._version for t in (x, z, h0, marks)]
    out, state = W.gated_forward(x, z, h0, checkpoints=marks)
    W.gated_backward(x, z, torch.ones_like(x), h0, h0, checkpoints=marks)
    W.gated_step(h0, x[:, 0], z[:, 0])
    assert [t._version for t in (x, z, h0, marks)] == v[:3] + [v[3] + 1]
    assert out._version == state._version == 0
    with torch.inference_mode():
        h = h0.clone()
        before = h.clone()
        W.gated_step(h, x[:, 0], z[:, 0], inplace=True)
    W.gated_step(h, x[:, 0], z[:, 0], inplace=True)
    assert not torch.equal(h, before)


def test_a_wait_that_runs_out_on_the_kept_workspace_is_reported():
    """The same where the caller passes no workspace: the status of the one that is kept for the stream can be queried, and
    is carried on when a larger one takes its place."""
    from wkv_recurrence_b200._native import ext
    with torch.cuda.stream(torch.cuda.Stream()):
        assert W.gated_status() == 0  # none is kept yet
        x = torch.randn(1, 260, 64, device="cuda")
        W.gated_forward(x, x)
        assert W.gated_status() == 0
        small = ext().gated_kept_workspace(torch.cuda.current_device())
        assert small.numel() >= W.gated_workspace_size(1, 260, 64)
        for grow in (False, True):
            small[:4].view(torch.int32).fill_(1)  # the ticket of tile 0 is gone: its total never arrives
            W.gated_forward(x, x)
            if grow:
                tiles = small.numel() // (8 * 64 * 16) + 1  # 16 bytes for each of 64 channels of 8 groups, and more
                W.gated_forward(*[torch.zeros(2, 128 * tiles, 256, device="cuda")] * 2)
                assert ext().gated_kept_workspace(torch.cuda.current_device()).numel() > small.numel()
            assert W.gated_status(torch.cuda.current_device()) == 6  # WKV_ERR_WAIT_TIMEOUT
            assert W.gated_status("cuda") == 0
        out, state = W.gated_forward(x, x)
        assert W.gated_status() == 0
        check_forward(x, x, None, "sigmoid", out, state)


def test_a_call_under_a_torch_mode_leaves_no_trace():
    """A call that is refused because its tensors hold no data, and a call under a mode that replaces what torch's operators
    return, do not spoil the workspace kept for the calls after them."""
    from torch._subclasses.fake_tensor import FakeTensorMode

    x, z, h0 = draw(2, 300, 64, F32, F32, "sigmoid")
    want = W.gated_forward(x, z, h0)
    with torch.cuda.stream(torch.cuda.Stream()):
        with FakeTensorMode() as mode:
            fake = mode.from_tensor(x)
            with pytest.raises(RuntimeError):
                W.gated_forward(fake, fake)
            inside = W.gated_forward(x, z, h0)
        after = W.gated_forward(x, z, h0)
        torch.cuda.current_stream().synchronize()
    for got in (inside, after):
        assert type(got[0]) is torch.Tensor and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_step_in_place_takes_no_other_state_out():
    x, z, h0 = draw(3, 1, 64, F32, F32, "sigmoid")
    x, z, other = x[:, 0], z[:, 0], torch.zeros_like(h0)
    with pytest.raises(ValueError, match="inplace"):
        W.gated_step(h0, x, z, state_out=other, inplace=True)
    want = W.gated_step(h0, x, z)
    for inplace in (False, True):
        s = h0.clone()
        out, state = W.gated_step(s, x, z, state_out=s, inplace=inplace)
        assert state is s and torch.equal(state, want[1]) and torch.equal(out, want[0])


@pytest.mark.parametrize("gate", ["sigmoid", "decay"])
@pytest.mark.parametrize("xt,zt,ot", TYPES)
@pytest.mark.parametrize("C", [64, 128, 768])
@pytest.mark.parametrize("T", [129, 517, 1024])
def test_whole_tiles_of_every_type(T, C, xt, zt, ot, gate):
    """Rows of 16-byte copies, channel groups of 64 and spans that are full."""
    x, z, h0 = draw(2, T, C, xt, zt, gate, seed=3)
    marks = W.gated_checkpoints(x)
    out, state = W.gated_forward(x, z, h0, gate=gate, out_dtype=ot, checkpoints=marks)
    g, ds = torch.randn(2, T, C, device="cuda").to(ot), torch.randn(2, C, device="cuda")
    got = W.gated_backward(x, z, g, h0, ds, gate=gate, checkpoints=marks)
    check_forward(x, z, h0, gate, out, state)
    check_backward(x, z, h0, g, ds, gate, got)


@pytest.mark.parametrize("gate", ["sigmoid", "decay"])
@pytest.mark.parametrize("xt,zt,ot", TYPES)
def test_many_channel_groups_of_every_type(xt, zt, ot, gate):
    """256 channel groups and more: every tile takes the state from the one before it (look-back groups of one)."""
    B, T, C = 33, 400, 512
    x, z, h0 = draw(B, T, C, xt, zt, gate, seed=4)
    marks = W.gated_checkpoints(x)
    out, state = W.gated_forward(x, z, h0, gate=gate, out_dtype=ot, checkpoints=marks)
    g, ds = torch.randn(B, T, C, device="cuda").to(ot), torch.randn(B, C, device="cuda")
    got = W.gated_backward(x, z, g, h0, ds, gate=gate, checkpoints=marks)
    for row, cols in ((0, slice(0, 130)), (17, slice(190, 258)), (B - 1, slice(C - 70, C))):
        cut = lambda t: t[row:row + 1, ..., cols].contiguous()  # noqa: E731
        check_forward(cut(x), cut(z), cut(h0), gate, cut(out), cut(state))
        check_backward(cut(x), cut(z), cut(h0), cut(g), cut(ds), gate, [cut(t) for t in got])


@pytest.mark.parametrize("gate,starts,slow", [("sigmoid", False, False), ("sigmoid", True, False), ("decay", False, True),
                                              ("decay", True, False)])
@pytest.mark.parametrize("size", [1e12, 1e30])
@pytest.mark.parametrize("B,C", [(1, 64), (50, 40)])
def test_large_states(B, C, size, gate, starts, slow):
    """States far above 2^32, fast and slow gates: as small ones, at their scale."""
    x, z, h0 = draw(B, 128 * 40 + 17, C, F32, F32, gate, seed=6, starts=starts, slow=slow)
    x, h0 = size * x, size * h0
    marks = W.gated_checkpoints(x)
    out, state = W.gated_forward(x, z, h0, gate=gate, checkpoints=marks)
    g, ds = torch.randn_like(x), torch.randn_like(h0)
    got = W.gated_backward(x, z, g / size, h0, ds / size, gate=gate, checkpoints=marks)
    for row in {0, B - 1}:
        cut = lambda t: t[row:row + 1, ..., C - 9:].contiguous()  # noqa: E731
        check_forward(cut(x), cut(z), cut(h0), gate, cut(out), cut(state))
        check_backward(cut(x), cut(z), cut(h0), cut(g / size), cut(ds / size), gate, [cut(t) for t in got])
