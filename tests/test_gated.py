"""The gated linear recurrence without a GPU: what the entry points refuse, and
the oracle against itself."""
import ctypes

import numpy as np
import pytest
import torch

import wkv_recurrence_b200 as W
from oracle import gated_oracle as G
from wkv_recurrence_b200 import _abi
from wkv_recurrence_b200 import build as wbuild

F32, BF16 = _abi.WKV_F32, _abi.WKV_BF16
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    wbuild.build()
    wbuild.build_ext()
    return _abi.lib()


def fwd(L, B=1, T=10, C=4, x=P(256), xt=F32, xs=(40, 4), z=P(256), zt=F32, zs=(40, 4), gate=0, out=P(256), ot=F32,
        ws=None, nws=0):
    return L.wkv_gated_forward(B, T, C, x, xt, *xs, z, zt, *zs, gate, out, ot, None, None, None, ws, nws, None)


def bwd(L, B=1, T=10, C=4, x=P(256), xt=F32, z=P(256), zt=F32, gate=0, g=P(256), gt=F32, marks=None, dx=P(256), dz=P(256),
        ws=None, nws=0):
    return L.wkv_gated_backward(B, T, C, x, xt, T * C, C, z, zt, T * C, C, gate, g, gt, None, None, marks, dx, dz, None, ws,
                                nws, None)


def test_workspace_size(L):
    assert L.wkv_gated_workspace_size(1, 128, 64) == 256  # one tile: nothing travels
    a, b = L.wkv_gated_workspace_size(2, 1000, 96), L.wkv_gated_workspace_size(2, 4000, 96)
    assert 256 < a < b
    for bad in ((-1, 1, 1), (1, 1 << 24, 1), (1, 1, 1 << 31), (1 << 20, 1 << 23, 1 << 12)):
        assert L.wkv_gated_workspace_size(*bad) == 0
    with pytest.raises(ValueError):
        W.gated_workspace_size(-1, 2, 3)
    text = open(wbuild.HEADER).read()
    assert f"#define WKV_GATED_TILE {_abi.WKV_GATED_TILE}\n" in text


def test_refusals_before_any_launch(L):
    E = _abi
    assert fwd(L, B=-1) == E.WKV_ERR_INVALID_ARG
    assert fwd(L, T=1 << 24) == E.WKV_ERR_INVALID_ARG
    assert fwd(L, gate=2) == E.WKV_ERR_INVALID_ARG
    assert fwd(L, xs=(40, -4)) == E.WKV_ERR_INVALID_ARG
    assert fwd(L, T=3, zs=(0, (1 << 62))) == E.WKV_ERR_INVALID_ARG
    assert fwd(L, x=None) == E.WKV_ERR_INVALID_ARG
    assert fwd(L, xt=7) == E.WKV_ERR_UNSUPPORTED_DTYPE
    assert fwd(L, xt=F32, zt=BF16) == E.WKV_ERR_UNSUPPORTED_DTYPE
    assert fwd(L, xt=F32, ot=BF16) == E.WKV_ERR_UNSUPPORTED_DTYPE
    assert fwd(L, x=P(258)) == E.WKV_ERR_MISALIGNED
    assert fwd(L, xt=BF16, ot=BF16, out=P(257)) == E.WKV_ERR_MISALIGNED
    assert fwd(L, T=129) == E.WKV_ERR_INVALID_ARG  # several tiles need a workspace
    n = L.wkv_gated_workspace_size(1, 129, 4)
    assert fwd(L, T=129, ws=P(256), nws=n - 1) == E.WKV_ERR_WORKSPACE_TOO_SMALL
    assert fwd(L, T=129, ws=P(128), nws=n) == E.WKV_ERR_MISALIGNED
    assert bwd(L, g=None) == E.WKV_ERR_INVALID_ARG
    assert bwd(L, dz=None) == E.WKV_ERR_INVALID_ARG
    assert bwd(L, xt=BF16, zt=F32, gt=BF16, g=P(257)) == E.WKV_ERR_MISALIGNED
    assert bwd(L, T=129, ws=P(256), nws=n) == E.WKV_ERR_INVALID_ARG  # several tiles need the checkpoints
    assert bwd(L, T=129, ws=P(256), nws=n - 1, marks=P(256)) == E.WKV_ERR_WORKSPACE_TOO_SMALL
    assert L.wkv_gated_step(2, 4, P(256), F32, 4, P(256), F32, 4, 0, P(256), F32, None, P(256), None) == \
        E.WKV_ERR_INVALID_ARG
    assert L.wkv_gated_step(2, 4, P(256), F32, -4, P(256), F32, 4, 0, P(256), F32, P(256), P(256), None) == \
        E.WKV_ERR_INVALID_ARG
    assert L.wkv_gated_step(1 << 30, 1 << 20, None, F32, 4, None, F32, 4, 0, None, F32, None, None, None) == \
        E.WKV_ERR_INVALID_ARG


def test_binding_refuses_cpu_tensors_and_names_the_argument(L):
    x = torch.zeros(1, 2, 3)
    for call in (lambda: W.gated_forward(x, x), lambda: W.gated_backward(x, x, x),
                 lambda: W.gated_step(x[0], x[0], x[0]), lambda: W.Gated.apply(x, x)):
        with pytest.raises(ValueError, match="x must be a CUDA tensor"):
            call()


@pytest.mark.parametrize("gate", ["sigmoid", "decay"])
def test_oracle_gradients_are_the_forwards_differences(gate):
    rng = np.random.default_rng(3)
    x, h0 = rng.normal(size=(2, 6, 3)), rng.normal(size=(2, 3))
    z = rng.normal(size=x.shape) if gate == "sigmoid" else np.exp(rng.normal(size=x.shape))
    g, ds = rng.normal(size=x.shape), rng.normal(size=h0.shape)
    loss = lambda a: sum(float((u * v).sum()) for u, v in zip(G.forward(*a, gate), (g, ds)))  # noqa: E731
    args = [x, z, h0]
    for k, grad in enumerate(G.backward(x, z, h0, g, ds, gate)):
        for at in np.ndindex(grad.shape):
            up, down = [a.copy() for a in args], [a.copy() for a in args]
            up[k][at] += 1e-5
            down[k][at] -= 1e-5
            assert abs((loss(up) - loss(down)) / 2e-5 - grad[at]) < 1e-8


@pytest.mark.parametrize("gate", ["sigmoid", "decay"])
def test_oracle_bound_holds_for_an_fp32_evaluation_and_catches_a_wrong_gate(gate):
    """The running error bound covers the recurrence in numpy's fp32, and does not cover a gate off by 1e-3."""
    rng = np.random.default_rng(4)
    x = rng.normal(size=(1, 400, 16)).astype(np.float32)
    z = (rng.normal(size=x.shape) if gate == "sigmoid" else np.exp(rng.normal(-2, 1, size=x.shape))).astype(np.float32)
    ref, _ = G.forward(x, z, None, gate)
    al, _ = G.allowed_forward(x, z, None, gate)
    for off in (0, 1e-3):
        f = (1 / (1 + np.exp(-z)) if gate == "sigmoid" else np.exp(-z)).astype(np.float32) * np.float32(1 - off)
        i = (1 / (1 + np.exp(z))).astype(np.float32) if gate == "sigmoid" else np.ones_like(f)
        h = np.zeros((1, 16), np.float32)
        worst = 0.0
        for t in range(400):
            h = f[:, t] * h + i[:, t] * x[:, t]
            worst = max(worst, float(((np.abs(h - ref[:, t]) - np.abs(ref[:, t]) * 2.0 ** -24) / al[:, t]).max()))
        assert worst < 1 if off == 0 else worst > 1


def test_gated_status_is_offered():
    assert "gated_status" in W.__all__
    with pytest.raises((ValueError, RuntimeError)):
        W.gated_status("cpu")


def test_states_off_four_bytes_are_refused(L):
    """A state, checkpoint or gradient pointer that no float can be read from."""
    n = L.wkv_gated_workspace_size(1, 129, 4)
    for at in range(3):
        ptr = [None, None, P(256)]
        ptr[at] = P(258)
        assert L.wkv_gated_forward(1, 129, 4, P(256), F32, 516, 4, P(256), F32, 516, 4, 0, P(256), F32, *ptr, P(256), n - 1,
                                   None) == _abi.WKV_ERR_MISALIGNED
    for at in (0, 1, 2, 5):
        ptr = [None, None, P(256), P(256), P(256), None]  # state, dstate, checkpoints, dx, dz, dstate_in
        ptr[at] = P(257)
        assert L.wkv_gated_backward(1, 129, 4, P(256), F32, 516, 4, P(256), F32, 516, 4, 0, P(256), F32, *ptr, P(256), n - 1,
                                    None) == _abi.WKV_ERR_MISALIGNED
