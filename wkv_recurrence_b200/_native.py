"""Loads _wkv_torch.so, the native calling path of the gated recurrence and the
RMS norm (csrc/wkv_torch.cpp), and binds it to the library that _abi loaded.
Fails loudly if it has not been built, or was built against another torch or
interpreter; there is no other path.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

from . import _abi

PATH = os.path.join(_abi.HERE, "_build", "_wkv_torch.so")
_ENTRIES = ("wkv_gated_workspace_size", "wkv_gated_forward", "wkv_gated_backward", "wkv_gated_step", "wkv_rms_norm",
            "wkv_rms_norm_quant", "wkv_rms_norm_backward_workspace_size", "wkv_rms_norm_backward")
_ext = None


def ext():
    global _ext
    if _ext is None:
        if not os.path.exists(PATH):
            raise RuntimeError(f"_wkv_torch.so is not built ({PATH}); run python -m wkv_recurrence_b200.build")
        lib = _abi.lib()
        spec = importlib.util.spec_from_file_location("_wkv_torch", PATH)
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        from . import build
        if mod.built_for() != build.ext_key():
            raise RuntimeError(f"_wkv_torch.so is built for {mod.built_for()}, and this is {build.ext_key()}; "
                               "run python -m wkv_recurrence_b200.build")
        mod.bind({n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _ENTRIES}, _abi.check,
                 torch.OutOfMemoryError)
        _ext = mod
    return _ext
