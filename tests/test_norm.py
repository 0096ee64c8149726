"""The RMS norm without a GPU: what the entry points refuse, and the oracle
against itself."""
import ctypes

import numpy as np
import pytest
import torch

import wkv_recurrence_b200 as W
from oracle import norm_oracle as R
from wkv_recurrence_b200 import _abi
from wkv_recurrence_b200 import build as wbuild

F32, BF16 = _abi.WKV_F32, _abi.WKV_BF16
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    wbuild.build()
    wbuild.build_ext()
    return _abi.lib()


def fwd(L, N=2, C=64, groups=1, eps=1e-6, x=P(256), xt=F32, xs=64, res=None, rt=F32, rs=64, w=P(256), y=P(256), yt=F32, s=None):
    return L.wkv_rms_norm(N, C, groups, eps, x, xt, xs, res, rt, rs, w, y, yt, s, None)


def quant(L, C=64, block=0, scale=P(256)):
    return L.wkv_rms_norm_quant(2, C, 1, 1e-6, P(256), F32, C, None, F32, 0, P(256), P(256), scale, block, None, None)


def bwd(L, N=2, C=64, groups=1, eps=1e-6, gy=P(256), gt=F32, s=P(256), st=F32, w=P(256), gs=None, ds=P(256), dw=P(256),
        ws=P(256), nws=None):
    nws = L.wkv_rms_norm_backward_workspace_size(N, C, groups) if nws is None else nws
    return L.wkv_rms_norm_backward(N, C, groups, eps, gy, gt, s, st, C, w, gs, ds, dw, ws, nws, None)


def test_refusals_before_any_launch(L):
    E = _abi
    for bad in (dict(N=-1), dict(C=-8), dict(groups=0), dict(groups=3), dict(C=16384, groups=16384, xs=16384), dict(eps=0.0),
                dict(eps=float("nan")), dict(xs=-1), dict(x=None), dict(w=None), dict(y=None), dict(res=P(256)),
                dict(N=1 << 31), dict(C=1 << 24)):
        assert fwd(L, **bad) == E.WKV_ERR_INVALID_ARG, bad
    for bad in (dict(xt=5), dict(yt=BF16), dict(yt=3), dict(res=P(256), s=P(256), rt=BF16), dict(res=P(256), s=P(256), rt=9)):
        assert fwd(L, **bad) == E.WKV_ERR_UNSUPPORTED_DTYPE, bad
    for bad in (dict(x=P(258)), dict(w=P(257)), dict(y=P(2)), dict(res=P(6), s=P(256)), dict(res=P(256), s=P(2))):
        assert fwd(L, **bad) == E.WKV_ERR_MISALIGNED, bad
    assert quant(L, block=16) == E.WKV_ERR_INVALID_ARG
    assert quant(L, block=-32) == E.WKV_ERR_INVALID_ARG
    assert quant(L, C=96, block=64) == E.WKV_ERR_INVALID_ARG
    assert quant(L, scale=None) == E.WKV_ERR_INVALID_ARG
    assert quant(L, scale=P(2)) == E.WKV_ERR_MISALIGNED
    for bad in (dict(groups=3), dict(eps=-1.0), dict(gy=None), dict(s=None), dict(w=None), dict(ds=None), dict(dw=None),
                dict(ws=None, nws=1 << 30)):
        assert bwd(L, **bad) == E.WKV_ERR_INVALID_ARG, bad
    assert bwd(L, st=BF16) == E.WKV_ERR_UNSUPPORTED_DTYPE
    assert bwd(L, nws=255) == E.WKV_ERR_WORKSPACE_TOO_SMALL
    assert bwd(L, ws=P(128)) == E.WKV_ERR_MISALIGNED
    assert bwd(L, gs=P(258)) == E.WKV_ERR_MISALIGNED
    assert L.wkv_rms_norm_backward_workspace_size(-1, 8, 1) == 0
    assert L.wkv_rms_norm_backward_workspace_size(4, 8, 3) == 0
    assert L.wkv_rms_norm_backward_workspace_size(4, 0, 1) == 256 == L.wkv_rms_norm_backward_workspace_size(0, 0, 1)


def test_binding_refuses_cpu_tensors_and_names_the_argument(L):
    x, w = torch.zeros(2, 8), torch.ones(8)
    for call, name in ((lambda: W.rms_norm(x, w), "x"), (lambda: W.rms_norm_quant(x, w), "x"),
                       (lambda: W.rms_norm_backward(x, x, w), "s"), (lambda: W.RMSNorm.apply(x, w), "x")):
        with pytest.raises(ValueError, match=f"{name} must be a CUDA tensor"):
            call()


def test_oracle_gradients_are_the_norms_differences():
    rng = np.random.default_rng(1)
    s, w, gy, gs = rng.normal(size=(3, 12)), rng.normal(size=12), rng.normal(size=(3, 12)), rng.normal(size=(3, 12))
    ds, dw, *_ = R.backward(gy, s, w, gs, 1e-3, 4)
    loss = lambda a, b: float((R.rms(a, b, 1e-3, 4)[0] * gy).sum() + (a * gs).sum())  # noqa: E731
    for at in np.ndindex(s.shape):
        e = np.zeros_like(s)
        e[at] = 1e-6
        assert abs((loss(s + e, w) - loss(s - e, w)) / 2e-6 - ds[at]) < 1e-7
    for at in range(12):
        e = np.zeros(12)
        e[at] = 1e-6
        assert abs((loss(s, w + e) - loss(s, w - e)) / 2e-6 - dw[at]) < 1e-7


def test_oracle_bound_holds_for_an_fp32_evaluation_and_catches_a_wrong_eps():
    rng = np.random.default_rng(2)
    s, w, gy = (rng.normal(size=n).astype(np.float32) for n in ((20, 96), 96, (20, 96)))
    want, wdw, bound, dwb = R.backward(gy, s, w, None, 1e-6, 2)
    for eps, ok in ((1e-6, True), (1e-3, False)):
        h, p = s.reshape(20, 2, 48), (gy * w).reshape(20, 2, 48)
        r = 1 / np.sqrt((h * h).mean(-1, keepdims=True, dtype=np.float32) + np.float32(eps))
        ds = (r * (p - h * (p * h).mean(-1, keepdims=True) * r * r)).reshape(20, 96)
        dw = (gy * (h * r).reshape(20, 96)).sum(0)
        assert (np.abs(ds - want) <= bound + np.abs(want) * 2.0 ** -24).all() == ok
        assert (np.abs(dw - wdw) <= dwb).all() == ok
