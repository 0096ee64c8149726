"""Which builds of the native calling path are taken, and which are made anew."""
import os
import types

import pytest

from wkv_recurrence_b200 import _native
from wkv_recurrence_b200 import build as wbuild


@pytest.fixture
def compiler(tmp_path, monkeypatch):
    """build_ext into a folder of its own with a compiler that only writes the file asked for; the commands it got."""
    got = []

    def run(cmd, check):
        got.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(wbuild, "EXT", str(tmp_path / "_build" / "_wkv_torch.so"))
    monkeypatch.setattr(wbuild, "subprocess", types.SimpleNamespace(run=run))
    return got


def test_the_calling_path_is_built_anew_for_another_torch(compiler, monkeypatch):
    assert wbuild.build_ext() == wbuild.EXT and len(compiler) == 1
    wbuild.build_ext()
    assert len(compiler) == 1  # nothing changed
    key = wbuild.ext_key()
    assert f'-DWKV_EXT_KEY="{key}"' in compiler[0]
    monkeypatch.setattr(wbuild, "ext_key", lambda: key.replace("torch ", "torch 9."))
    wbuild.build_ext()
    assert len(compiler) == 2
    wbuild.build_ext()
    assert len(compiler) == 2
    os.remove(wbuild.EXT + ".key")  # an object whose key is not known
    wbuild.build_ext()
    assert len(compiler) == 3
    os.utime(wbuild.EXT, (0, 0))  # older than its source
    wbuild.build_ext()
    assert len(compiler) == 4


def test_an_object_for_another_torch_is_refused(monkeypatch):
    wbuild.build()
    wbuild.build_ext()
    monkeypatch.setattr(_native, "_ext", None)
    assert _native.ext().built_for() == wbuild.ext_key()
    monkeypatch.setattr(_native, "_ext", None)
    monkeypatch.setattr(wbuild, "ext_key", lambda: "torch 9")
    with pytest.raises(RuntimeError, match="this is torch 9"):
        _native.ext()
