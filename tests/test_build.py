"""The build's order and what it needs: the C library is there without PyTorch,
and whatever becomes of the Python binding's native module.  The compilers are
stand-ins that write their output file, so nothing is compiled here."""
import os
import sys

import pytest

from nvfp4_w4a4_block_quantize_amd import build as b
from nvfp4_w4a4_block_quantize_amd import kv


@pytest.fixture
def sandbox(tmp_path, monkeypatch):
    """build.py with its outputs under tmp_path and stand-in compilers."""
    good, bad = tmp_path / "compiler", tmp_path / "broken_compiler"
    good.write_text('#!/bin/sh\nwhile [ $# -gt 0 ]; do if [ "$1" = -o ]; then echo built > "$2"; fi; shift; done\n')
    bad.write_text("#!/bin/sh\necho no headers >&2\nexit 1\n")
    for f in (good, bad):
        f.chmod(0o755)
    outputs = dict(LIB_PATH="libnvfp4.so", BIND_PATH="_kv_bind.so", CONFORMANCE_PATH="conformance_cvt", PROBES_PATH="probes.so")
    for name, file in outputs.items():
        monkeypatch.setattr(b, name, str(tmp_path / file))
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "HIPCC", str(good))
    monkeypatch.setattr(b, "CXX", str(good))
    return tmp_path


COMPILED = {"libnvfp4.so", "conformance_cvt", "probes.so"}


def built(path):
    return set(os.listdir(path)) & (COMPILED | {"_kv_bind.so"})


def test_all_is_built_where_torch_is(sandbox):
    pytest.importorskip("torch")
    assert b.build() == b.LIB_PATH
    assert built(sandbox) == COMPILED | {"_kv_bind.so"}


def test_the_library_needs_no_torch(sandbox, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch fails
    (sandbox / "_kv_bind.so").write_text("of an earlier build")
    assert b.build(verbose=True) == b.LIB_PATH
    assert built(sandbox) == COMPILED  # no binding is left that belongs to another library


def test_the_library_is_there_when_the_binding_fails(sandbox, monkeypatch):
    pytest.importorskip("torch")
    monkeypatch.setattr(b, "CXX", str(sandbox / "broken_compiler"))
    with pytest.raises(RuntimeError, match="no headers"):
        b.build()
    assert built(sandbox) == COMPILED


def test_a_missing_binding_is_named(monkeypatch):
    torch = pytest.importorskip("torch")
    if not os.path.exists(b.LIB_PATH):
        pytest.skip("libnvfp4.so not built")
    monkeypatch.setitem(sys.modules, "nvfp4_w4a4_block_quantize_amd._kv_bind", None)
    monkeypatch.delattr("nvfp4_w4a4_block_quantize_amd._kv_bind", raising=False)
    monkeypatch.setattr(kv, "_bind", None)
    x = torch.zeros((1, 1, 64))
    with pytest.raises(RuntimeError, match="_kv_bind.so is missing"):
        kv.nvfp4_rope(x, None, torch.zeros((1, 1), dtype=torch.int32), torch.zeros(1), torch.zeros(1, dtype=torch.int32))
