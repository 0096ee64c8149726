"""The RMS norm on the GPU against its float64 oracle: types, groups, odd sizes
and alignments, e4m3 scales, gradients, strides, rows of zeros, and a run of it
with the gated recurrence."""
import numpy as np
import pytest
import torch

import wkv_recurrence_b200 as W
from oracle import gated_oracle as G
from oracle import norm_oracle as R

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
# half a step of the type, relative to the value
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
EPS = 1e-6
TYPES = [(F32, None, F32), (F32, F32, F32), (BF16, None, BF16), (BF16, BF16, BF16), (BF16, F32, BF16), (BF16, F32, F32)]


def np64(t):
    return t.detach().double().cpu().numpy()


def draw(N, C, xt, rt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(7 * N + C + seed)
    x = torch.randn(N, C, generator=g, device="cuda").to(xt)
    res = None if rt is None else (3 * torch.randn(N, C, generator=g, device="cuda")).to(rt)
    w = 1 + 0.2 * torch.randn(C, generator=g, device="cuda")
    return x, res, w


def check_y(y, s, w, groups, eps=EPS):
    ref, _ = R.rms(np64(s), np64(w), eps, groups)
    rel = R.rel_y(s.shape[1] // groups) + HALF[y.dtype]
    got = np64(y)
    assert got.shape == ref.shape
    bad = ~(np.abs(got - ref) <= rel * 1.01 * np.abs(ref) + 1e-37)
    assert not bad.any(), (int(bad.sum()), got[bad][:3], ref[bad][:3])
    return ref


def check_sum(s, x, res):
    want = (x.double() + res.double()).to(res.dtype)  # fp32 rounds a bf16 sum once more only far below half a step
    if res.dtype == F32:
        assert torch.equal(s, x.float() + res)
    else:
        d = (s.double() - want.double()).abs()
        assert bool((d <= 2.0 ** -8 * want.double().abs() * 2 ** -7).all())


SIZES = [(1, 1, 1), (3, 8, 1), (5, 64, 1), (2, 96, 1), (7, 100, 1), (4, 256, 2), (3, 768, 12), (9, 768, 8), (2, 1024, 1),
         (3, 1032, 1), (2, 4096, 1), (2, 4097, 1), (1, 16384, 1), (1, 20000, 1), (2, 40000, 1), (3, 60, 3), (2, 51, 17),
         (2, 2048, 2), (5, 3200, 5), (1, 33000, 1), (65, 57, 1), (33, 250, 10), (9, 771, 1), (40, 1000, 8), (5, 201, 1)]


@pytest.mark.parametrize("N,C,groups", SIZES)
@pytest.mark.parametrize("xt,rt,yt", TYPES)
def test_forward(N, C, groups, xt, rt, yt):
    x, res, w = draw(N, C, xt, rt)
    y, s = W.rms_norm(x, w, res, groups=groups, out_dtype=yt)
    assert y.dtype == yt
    if res is None:
        assert s is None
        s = x
    else:
        check_sum(s, x, res)
    check_y(y, s, w, groups)


def check_q(q, scale, s, w, groups, block):
    y, _ = R.rms(np64(s), np64(w), EPS, groups)
    want = R.scales(y, block)
    rel = R.rel_y(s.shape[1] // groups)
    sc = np64(scale)
    assert sc.shape == want.shape
    assert (np.abs(sc - want) <= want * (rel + 2 * 2.0 ** -24) + 1e-37).all()
    N, C = y.shape
    b = block or C
    back = np64(q.float()).reshape(N, C // b, b) * sc[..., None]
    ratio = np.abs(y.reshape(N, C // b, b)) / sc[..., None]
    # half a step of e4m3: 2^-4 of the value, or 2^-10 (half of the subnormal step 2^-9) below 2^-6
    lim = np.maximum(ratio * 2.0 ** -4, 2.0 ** -10) * sc[..., None]
    err = np.abs(back - y.reshape(N, C // b, b))
    assert (err <= lim * 1.0001 + np.abs(y.reshape(N, C // b, b)) * rel * 2 + 1e-37).all()


@pytest.mark.parametrize("N,C,groups,block", [(1, 1, 1, 0), (5, 64, 1, 0), (5, 64, 1, 32), (3, 100, 1, 0), (4, 96, 1, 32),
                                              (7, 768, 12, 64), (7, 768, 12, 0), (7, 768, 12, 128), (3, 768, 8, 32),
                                              (2, 1152, 12, 128), (3, 128, 1, 128), (2, 128, 4, 128), (2, 4096, 1, 0),
                                              (2, 4096, 1, 128), (1, 20480, 1, 128), (1, 40000, 1, 0), (2, 384, 1, 128),
                                              (2, 640, 1, 64), (2, 512, 2, 128), (3, 4128, 1, 32), (1, 256, 32, 0)])
@pytest.mark.parametrize("xt,rt", [(F32, None), (BF16, BF16), (BF16, F32)])
def test_quant(N, C, groups, block, xt, rt):
    x, res, w = draw(N, C, xt, rt)
    q, scale, s = W.rms_norm_quant(x, w, res, groups=groups, block=block)
    assert q.dtype == torch.float8_e4m3fn and scale.shape == (N, C // block if block else 1)
    check_q(q, scale, x if res is None else s, w, groups, block)


def test_rows_and_blocks_of_zeros():
    x, _, w = draw(4, 256, BF16, None)
    x[1] = 0
    x[2, 128:] = 0
    y, _ = W.rms_norm(x, w)
    assert torch.equal(y[1], torch.zeros_like(y[1]))
    for C in (256, 255):
        q, scale, _ = W.rms_norm_quant(x[:, :C].contiguous(), w[:C].contiguous(), block=0)
        assert float(scale[1]) == 1 and torch.equal(q[1].float(), torch.zeros(C, device="cuda"))
    q, scale, _ = W.rms_norm_quant(x, w, block=128)
    assert float(scale[2, 1]) == 1 and float(scale[2, 0]) != 1
    assert torch.equal(q[2, 128:].float(), torch.zeros(128, device="cuda"))
    # a row whose y is far below fp32's smallest normal number still has a finite inverse scale
    q, scale, _ = W.rms_norm_quant(torch.full((1, 64), 1e-38, device="cuda"), torch.full((64,), 1e-6, device="cuda"), eps=1.0)
    assert bool(scale.isfinite().all()) and bool((q.float() >= 0).all()) and float(scale) >= 1.17549435e-38
    # nor do zeros beside such values become anything else (1 / sqrt(eps) = 1000 on top of that inverse)
    x = torch.zeros(1, 64, device="cuda")
    x[0, ::2] = 2e-38
    for C in (64, 63):
        q, scale, _ = W.rms_norm_quant(x[:, :C].contiguous(), torch.full((C,), 1e-3, device="cuda"))
        assert bool((q.float()[0, 1::2] == 0).all()) and bool((q.float()[0, ::2] > 0).all())
    # squares that overflow: the norm is 0, as the formula's in fp32
    y, _ = W.rms_norm(torch.full((1, 64), 1e20, device="cuda"), torch.ones(64, device="cuda"))
    assert torch.equal(y, torch.zeros_like(y))


@pytest.mark.parametrize("N,C,groups", SIZES + [(700, 768, 12), (3001, 96, 1), (1500, 2048, 1), (400, 100, 5)])
@pytest.mark.parametrize("yt,st", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("with_gs", [False, True])
def test_backward(N, C, groups, yt, st, with_gs):
    gy, s, w = draw(N, C, yt, st, seed=5)
    gs = torch.randn(N, C, device="cuda").to(st) if with_gs else None
    ds, dw = W.rms_norm_backward(gy, s, w, gs, groups=groups)
    want, wdw, bound, dwb = R.backward(np64(gy), np64(s), np64(w), None if gs is None else np64(gs), EPS, groups)
    assert ds.dtype == st and dw.dtype == F32
    lim = bound + (np.abs(want) + bound) * HALF[st] + 1e-37
    assert (np.abs(np64(ds) - want) <= lim).all()
    assert (np.abs(np64(dw) - wdw) <= dwb + 1e-37).all()
    again = W.rms_norm_backward(gy, s, w, gs, groups=groups)
    assert torch.equal(again[0], ds) and torch.equal(again[1], dw)


def test_strides_shapes_and_in_place():
    big = torch.randn(3, 5, 2 * 72 + 3, device="cuda").to(BF16)
    w = torch.rand(72, device="cuda") + 0.5
    for x in (big[..., :72], big[..., 8:80], big[..., 1:73]):
        y, _ = W.rms_norm(x, w)
        assert y.shape == x.shape
        check_y(y.reshape(15, 72), x.reshape(15, 72), w, 1)
        ds, dw = W.rms_norm_backward(y, x, w)
        d2, w2 = W.rms_norm_backward(y, x.contiguous(), w)
        want, wdw, bound, dwb = R.backward(np64(y.reshape(15, 72)), np64(x.reshape(15, 72)), np64(w), None, EPS, 1)
        for a, b in ((ds, dw), (d2, w2)):
            assert (np.abs(np64(a.reshape(15, 72)) - want) <= bound + (np.abs(want) + bound) * HALF[BF16]).all()
            assert (np.abs(np64(b) - wdw) <= dwb).all()
    with pytest.raises(ValueError, match="one stride"):
        W.rms_norm(big.transpose(0, 1)[..., :72], w)
    for C in (72, 71):
        x, res, w = draw(6, C, BF16, F32)
        want, s = W.rms_norm(x, w, res)
        y, s2 = W.rms_norm(x, w, res, residual_out=res)
        assert s2 is res and torch.equal(s2, s) and torch.equal(y, want)
    y, _ = W.rms_norm(big[0, 0, :72], w[:1].expand(72).contiguous())
    assert y.shape == (72,)


def test_empty():
    w = torch.ones(8, device="cuda")
    e = torch.empty(0, 8, device="cuda")
    assert W.rms_norm(e, w, e)[0].shape == (0, 8)
    assert W.rms_norm_quant(e, w)[1].shape == (0, 1)
    ds, dw = W.rms_norm_backward(e, e, w)
    assert ds.shape == (0, 8) and torch.equal(dw, torch.zeros_like(w))
    e = torch.empty(3, 0, device="cuda")
    assert W.rms_norm(e, w[:0])[0].shape == (3, 0)
    assert W.rms_norm_backward(e, e, w[:0])[1].shape == (0,)


def test_autograd_and_differences():
    x, res, w = draw(3, 40, F32, F32)
    x, res, w = (t.requires_grad_() for t in (x, res, w))
    y, s = W.RMSNorm.apply(x, w, res, EPS, 2)
    g, gs = torch.randn_like(y), torch.randn_like(s)
    dx, dw, dr = torch.autograd.grad((y * g).sum() + (s * gs).sum(), (x, w, res))
    assert torch.equal(dx, dr)

    def loss(a):
        t = a[0] + a[2]
        return float((R.rms(t, a[1], EPS, 2)[0] * np64(g)).sum() + (t * np64(gs)).sum())

    args = [np64(t) for t in (x, w, res)]
    rng = np.random.default_rng(0)
    for k, grad in enumerate((dx, dw, dr)):
        for _ in range(6):
            at = tuple(rng.integers(0, n) for n in args[k].shape)
            up, down = [a.copy() for a in args], [a.copy() for a in args]
            up[k][at] += 1e-5
            down[k][at] -= 1e-5
            want = (loss(up) - loss(down)) / 2e-5
            assert abs(float(grad[at]) - want) < 1e-5 * max(1, abs(want)) + 1e-6 * 10
    # a residual stream in fp32 beside bf16 activations; the stream's reader alone gives a gradient
    x, res, w = draw(4, 64, BF16, F32)
    x.requires_grad_(), res.requires_grad_()
    y, s = W.RMSNorm.apply(x, w, res)
    s.sum().backward()
    assert torch.equal(res.grad, torch.ones_like(res)) and torch.equal(x.grad, torch.ones_like(x))
    x2 = x.detach().clone().requires_grad_()
    W.RMSNorm.apply(x2, w).float().sum().backward()
    want = R.backward(np.ones((4, 64)), np64(x2), np64(w), None, EPS, 1)
    assert (np.abs(np64(x2.grad) - want[0]) <= want[2] + (np.abs(want[0]) + want[2]) * HALF[BF16]).all()


def test_many_rows():
    x, res, w = draw(70001, 64, BF16, BF16)
    y, s = W.rms_norm(x, w, res)
    for part in (slice(0, 100), slice(69901, 70001)):
        check_y(y[part], s[part], w, 1)


def test_captured_and_replayed():
    x, res, w = draw(33, 768, BF16, BF16)
    gy = torch.randn(33, 768, device="cuda").to(BF16)
    y, s = W.rms_norm(x, w, res)
    want = (y, s, *W.rms_norm_quant(x, w, res, block=128)[:2], *W.rms_norm_backward(gy, s, w))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, s = W.rms_norm(x, w, res)
        got = (y, s, *W.rms_norm_quant(x, w, res, block=128)[:2], *W.rms_norm_backward(gy, s, w))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.float(), b.float())


def test_a_layer_of_them():
    """Norm, projections to input and gate, gated recurrence, norm with the residual, 8 bits; and the gradients of
    the norm, recurrence, norm chain against float64."""
    B, T, C = 2, 200, 96
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(B, T, C, generator=g, device="cuda")
    w1, w2 = (1 + 0.1 * torch.randn(C, generator=g, device="cuda") for _ in range(2))
    proj = torch.randn(C, 2 * C, generator=g, device="cuda") / C ** 0.5
    y, _ = W.rms_norm(x, w1)
    both = y @ proj
    out, _ = W.gated_forward(both[..., :C], both[..., C:])  # the two halves as they lie
    z, s = W.rms_norm(out, w2, x, groups=8)
    q, scale, s2 = W.rms_norm_quant(out, w2, x, groups=8, block=32)
    assert torch.equal(s, s2) and torch.equal(s, out + x)
    ref, _ = G.forward(np64(both[..., :C]), np64(both[..., C:]), None, "sigmoid")
    al, _ = G.allowed_forward(np64(both[..., :C]), np64(both[..., C:]), None, "sigmoid")
    assert (np.abs(np64(out) - ref) <= (np.abs(ref) + al) * 2.0 ** -24 + al).all()
    check_y(z.reshape(-1, C), s.reshape(-1, C), w2, 8)
    check_q(q.reshape(-1, C), scale.reshape(-1, C // 32), s.reshape(-1, C), w2, 8, 32)

    leaves = [t.clone().requires_grad_() for t in (x, w1, w2)]
    y = W.RMSNorm.apply(leaves[0], leaves[1], None, EPS, 1)
    h, _ = W.Gated.apply(y, y * 0.5, None, "sigmoid")
    z, s = W.RMSNorm.apply(h, leaves[2], leaves[0], EPS, 8)
    gz = torch.randn(z.shape, generator=g, device="cuda")
    got = torch.autograd.grad((z * gz).sum(), leaves)

    d = [t.detach().double().cpu().requires_grad_() for t in (x, w1, w2)]
    norm = lambda t, w, k: (t.view(B, T, k, -1) * (t.view(B, T, k, -1).square().mean(-1, keepdim=True) + EPS).rsqrt()).reshape(B, T, C) * w  # noqa: E731
    y = norm(d[0], d[1], 1)
    f = torch.sigmoid(y * 0.5)
    hs, hh = [], torch.zeros(B, C, dtype=torch.float64)
    for t in range(T):
        hh = f[:, t] * hh + (1 - f[:, t]) * y[:, t]
        hs.append(hh)
    z = norm(torch.stack(hs, 1) + d[0], d[2], 8)
    want = torch.autograd.grad((z * gz.double().cpu()).sum(), d)
    # three operators in a row, each within about 1e-6 of its scale (see their own tests), amplified by at most the
    # norms' r ~ 1 and summed over 400 rows for the weights
    for a, b in zip(got, want):
        assert float((a.double().cpu() - b).norm() / b.norm()) < 1e-5


def test_the_binding_refuses_on_the_gpu():
    x, w = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    bad = [(lambda: W.rms_norm(x, w[:8]), ValueError), (lambda: W.rms_norm(x, w.bfloat16()), TypeError),
           (lambda: W.rms_norm(x.half(), w), TypeError), (lambda: W.rms_norm(x, w.cpu()), ValueError),
           (lambda: W.rms_norm(x, w, x[:2]), ValueError), (lambda: W.rms_norm(x, w, x.bfloat16()), TypeError),
           (lambda: W.rms_norm(x, w, eps=0), ValueError), (lambda: W.rms_norm(x, w, eps=1e-60), ValueError),
           (lambda: W.rms_norm(x, w, eps="a"), TypeError), (lambda: W.rms_norm(x, w, groups=3), ValueError),
           (lambda: W.rms_norm(x, w, groups=0), ValueError), (lambda: W.rms_norm(x, w, out_dtype=BF16), TypeError),
           (lambda: W.rms_norm(x, w, residual_out=x), ValueError), (lambda: W.rms_norm(x.t(), w[:4]), ValueError),
           (lambda: W.rms_norm(torch.tensor(1.0, device="cuda"), w), ValueError),
           (lambda: W.rms_norm_quant(x, w, block=16), ValueError), (lambda: W.rms_norm_quant(x, w, block=128), ValueError),
           (lambda: W.rms_norm_backward(x, x.bfloat16(), w), TypeError), (lambda: W.rms_norm_backward(x[:2], x, w), ValueError),
           (lambda: W.rms_norm_backward(x, x, w, x.bfloat16()), TypeError),
           (lambda: W.rms_norm_backward(x, x, w, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda")), W.WkvError)]
    for call, kind in bad:
        with pytest.raises(kind):
            call()


@pytest.mark.parametrize("S,C", [(3, 64), (700, 768), (4096, 1024)])
def test_a_chain_of_calls_is_ordered(S, C):
    """Each call reads what the one before wrote, in place where that is allowed, with nothing between them: the kernels
    are launched before their predecessors end, and must not read before. The same calls with a wait between give the
    same bits."""
    g = torch.Generator(device="cuda").manual_seed(S)
    x0 = torch.randn(S, C, generator=g, device="cuda")
    w = 1 + 0.1 * torch.randn(C, generator=g, device="cuda")
    gates = torch.randn(S, C, generator=g, device="cuda")

    def run(wait):
        def after(*r):
            if wait:
                torch.cuda.synchronize()
            return r

        x, res, state = x0.clone(), x0.clone(), torch.zeros(S, C, device="cuda")
        kept = []
        for _ in range(12):
            y, res = after(*W.rms_norm(x, w, res, residual_out=res))
            x, state = after(*W.gated_step(state, y, gates, inplace=True))
            seq = torch.empty(2, S, C, device="cuda")
            h, last = after(*W.gated_forward(y.view(1, S, C), x.view(1, S, C), state[:1], out=seq[:1]))
            dx, dz, dh = after(*W.gated_backward(y.view(1, S, C), x.view(1, S, C), h, state[:1], last))
            x, dw = after(*W.rms_norm_backward(dx.view(S, C), h.view(S, C), w, dz.view(S, C)))
            q, scale, _ = after(*W.rms_norm_quant(x, w))
            kept += [x, dw, q.float(), scale, dh, state.clone()]
        torch.cuda.synchronize()
        return kept

    want = run(True)
    for _ in range(3):
        for a, b in zip(run(False), want):
            assert torch.equal(a, b)


def test_autograd_sees_what_was_written_in_place():
    """A backward whose saved s was overwritten raises, as behind torch's own in-place operators."""
    x, res, w = draw(6, 64, F32, F32)
    x.requires_grad_()
    for overwrite in (lambda s: W.rms_norm(x, w, s, residual_out=s), lambda s: W.rms_norm(x, w, out=s),
                      lambda s: W.rms_norm_quant(x, w, s, residual_out=s)):
        y, s = W.RMSNorm.apply(x, w, res)
        with torch.no_grad():
            overwrite(s)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
    v = [t._version for t in (x, res, w)]
    y, s = W.rms_norm(x, w, res)
    W.rms_norm_quant(x, w, res)
    W.rms_norm_backward(y, s, w, s)
    assert [t._version for t in (x, res, w, y, s)] == v + [0, 0]


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("C,groups,block,shift", [(512, 1, 128, 0), (512, 1, 0, 0), (768, 12, 64, 0), (768, 12, 128, 0),
                                                  (768, 12, 0, 0), (8192, 1, 128, 0), (768, 12, 128, 1), (2560, 5, 128, 0),
                                                  (100, 1, 0, 0)])
def test_quant_of_what_is_not_finite(C, groups, block, shift, bad):
    """A NaN or an infinity makes its group NaN (an infinity: itself alone, the others 0); it is NaN in q, and the scale is
    that of the block's other columns. Other rows do not notice."""
    x, _, w = draw(3, C + shift, F32, None)
    x, w = x[:, shift:], w[shift:].contiguous()
    x[1, C // groups + 3 if groups > 1 else 3] = bad
    q, scale, _ = W.rms_norm_quant(x, w, groups=groups, block=block)
    y, _ = W.rms_norm(x, w, groups=groups)
    assert bool(y[1].isnan().any()) and torch.equal(q.float().isnan(), y.isnan())
    b = block or C
    top = y[1].view(-1, b).nan_to_num(0.0).abs().amax(-1)
    want = torch.where(top > 0, top / 448, torch.ones_like(top))
    assert bool(((scale[1] - want).abs() <= want * 2.0 ** -20).all())
    good = q[1].float().view(-1, b) * scale[1][:, None]
    err = (good - y[1].view(-1, b)).nan_to_num(0.0).abs()
    assert bool((err <= top[:, None] * 2.0 ** -4 * 1.001).all())
    keep = torch.tensor([0, 2], device="cuda")
    check_q(q[keep], scale[keep], x[keep], w, groups, block)


@pytest.mark.parametrize("captured", [False, True])
def test_calls_that_wait_for_another_stream(captured):
    """A call behind an event of another stream reads what that stream's calls wrote, although it is launched before the
    call in front of it on its own stream ends; eager, and as the join of two branches of a graph."""
    N, C = 8192, 2048
    x, res, w = draw(N, C, F32, F32)
    gates = torch.randn(N, C, device="cuda")
    y0, s0 = W.rms_norm(x, w, res)
    small, _ = W.rms_norm(x[:16].contiguous(), w)
    want = W.gated_step(s0, y0, gates)
    wx, wdw = W.rms_norm_backward(want[0], want[1], w)
    torch.cuda.synchronize()
    other, mine = torch.cuda.Stream(), torch.cuda.Stream()
    y, s = torch.zeros_like(x), torch.zeros_like(x)
    head = torch.zeros_like(small)

    def run():
        fork, join = torch.cuda.Event(), torch.cuda.Event()
        fork.record()
        other.wait_event(fork)
        with torch.cuda.stream(other):
            for _ in range(3):
                W.rms_norm(x, w, res, out=y, residual_out=s)
            join.record()
        W.rms_norm(x[:16], w, out=head)
        torch.cuda.current_stream().wait_event(join)
        out, state = W.gated_step(s, y, gates)
        return (out, state, *W.rms_norm_backward(out, state, w))

    with torch.cuda.stream(mine):
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=mine):
                got = run()
        for _ in range(10):
            y.zero_()
            s.zero_()
            if captured:
                graph.replay()
            else:
                got = run()
            mine.synchronize()
            for a, b in zip(got, (*want, wx, wdw)):
                assert torch.equal(a, b)
            assert torch.equal(head, small)
