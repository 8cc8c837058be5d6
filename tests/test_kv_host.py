"""What the paged KV cache's C ABI layer decides on the host, with the launchers
and the HIP calls replaced (tests/abi_sanitize/kv_host_hooks.cpp)."""
import ctypes
import os
import shutil
import subprocess

import pytest

import nvfp4_w4a4_block_quantize_amd as nv
from tests.test_kv_abi import OK, REFUSED, SHAPE, P, calls

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "nvfp4_w4a4_block_quantize_amd", "csrc")
HOOKS = os.path.join(ROOT, "tests", "abi_sanitize", "kv_host_hooks.cpp")


@pytest.fixture(scope="module")
def host_lib(tmp_path_factory):
    rocm = next((p for p in (os.environ.get("ROCM_PATH"), "/opt/rocm")
                 if p and os.path.exists(os.path.join(p, "include", "hip", "hip_runtime.h"))), None)
    gxx = shutil.which("g++")
    if gxx is None or rocm is None or not os.path.exists(HOOKS):
        pytest.skip("needs g++, the HIP headers and the hooks' source")
    path = str(tmp_path_factory.mktemp("kv_host") / "libkv_host.so")
    cmd = [gxx, "-std=c++17", "-O1", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"),
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(CSRC, "nvfp4_kv_abi.cpp"), HOOKS, "-o", path]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    lib = ctypes.CDLL(path)
    for name, (res, args) in nv.KV_SIGNATURES.items():
        getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
    lib.kv_test_hip_calls.restype = ctypes.c_int64
    return lib


@pytest.mark.parametrize("change,copied", [
    ({}, (0, 10)),                                  # 8 query heads and 2 key heads
    ({"qo": P}, (8, 2)),                            # q in place: the keys alone
    ({"ko": P}, (0, 8)),
    ({"qo": P, "ko": P}, (8, 0)),
    ({"hk": 0, "k": None, "ko": None}, (0, 8)),
    ({"hk": 0, "k": None, "ko": None, "qo": P}, (8, 0))])
def test_rope_copies_no_head_that_is_turned_in_place(host_lib, change, copied):
    valid = dict(k=3 * P, ko=4 * P)
    change = {**valid, **{k: (3 * P if k == "ko" and v == P else v) for k, v in change.items()}}
    assert calls(host_lib)["rope"](**change) == OK
    first, count = ctypes.c_int32(-1), ctypes.c_int32(-1)
    host_lib.kv_test_rope_copied(ctypes.byref(first), ctypes.byref(count))
    assert (first.value, count.value) == copied


@pytest.mark.parametrize("op", sorted(REFUSED))
def test_refused_calls_ask_hip_nothing(host_lib, op):
    call, before = calls(host_lib)[op], host_lib.kv_test_hip_calls()
    for status, name, value in REFUSED[op]:
        assert call(**{name: value}) == status, (name, value)
        assert host_lib.kv_test_hip_calls() == before, (name, value)
    size = ctypes.c_int64(0)
    for heads in ((24, 4, 256), (7, 2, 64)):
        host_lib.nvfp4_paged_attention_workspace(*heads, ctypes.addressof(size))
    assert host_lib.kv_test_hip_calls() == before
    assert call() == OK and host_lib.kv_test_hip_calls() == before + 1


def test_the_workspace_is_wanted_to_the_byte(host_lib):
    call, size = calls(host_lib)["attend"], ctypes.c_int64(0)
    for hq, hk, dim in ((8, 2, 64), (24, 4, 256), (64, 1, 192), (32, 32, 128)):
        assert host_lib.nvfp4_paged_attention_workspace(hq, hk, dim, ctypes.addressof(size)) == OK
        heads = dict(hq=hq, hk=hk, dim=dim, qt=hq * dim, qh=dim, ot=hq * dim, oh=dim)
        assert call(**heads, bytes=size.value) == OK
        assert call(**heads, bytes=size.value - 1) == SHAPE


def test_one_row_of_positions_serves_all_axes(host_lib):
    call = calls(host_lib)["rope"]
    assert call(ld_pos=0) == OK and call(ld_pos=0, axes_n=1) == OK and call(ld_pos=4) == OK
    for bad in (-1, 1, 3, -(1 << 40)):
        assert call(ld_pos=bad) == SHAPE
