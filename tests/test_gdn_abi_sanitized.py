"""The gated delta layer's C ABI layer (csrc/nvfp4_gdn_abi.cpp) built for the host
alone with AddressSanitizer and UndefinedBehaviorSanitizer, its launchers
replaced by stubs, then the ctypes tests run against it in a child process; and,
of a plain build of the same files, that the workspace holds what calls use."""
import ctypes
import os
import random
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "nvfp4_w4a4_block_quantize_amd", "csrc")


def build(lib, *flags):
    rocm = next((p for p in (os.environ.get("ROCM_PATH"), "/opt/rocm")
                 if p and os.path.exists(os.path.join(p, "include", "hip", "hip_runtime.h"))), None)
    gxx = shutil.which("g++")
    if gxx is None or rocm is None:
        pytest.skip("needs g++ and the HIP headers")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fPIC", "-shared", *flags, "-D__HIP_PLATFORM_AMD__",
           "-I", os.path.join(rocm, "include"), "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(CSRC, "nvfp4_gdn_abi.cpp"), os.path.join(ROOT, "tests", "abi_sanitize", "gdn_launch_stubs.cpp"),
           "-o", lib, "-L", os.path.join(rocm, "lib"), "-lamdhip64", "-Wl,-rpath," + os.path.join(rocm, "lib")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]


def test_gdn_abi_layer_under_asan_and_ubsan(tmp_path):
    gxx = shutil.which("g++")
    asan = subprocess.run([gxx, "-print-file-name=libasan.so"], capture_output=True, text=True).stdout.strip() if gxx else ""
    if not os.path.isabs(asan) or not os.path.exists(asan):
        pytest.skip("no ASan runtime for g++")
    lib = str(tmp_path / "libnvfp4_gdn_abi_sanitized.so")
    build(lib, "-fno-omit-frame-pointer", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined")
    env = dict(os.environ, NVFP4_GDN_ABI_LIB=lib, NVFP4_NO_GPU="1", LD_PRELOAD=asan,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_gdn_abi.py"), "-k", "not binding"],
                       capture_output=True, text=True, env=env, cwd=ROOT, timeout=600)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "passed" in r.stdout and "ERROR: AddressSanitizer" not in r.stderr and "runtime error" not in r.stderr


def test_workspace_holds_what_a_call_and_smaller_calls_use(tmp_path):
    path = str(tmp_path / "libnvfp4_gdn_sizes.so")
    build(path)
    lib = ctypes.CDLL(path)
    i64, i32 = ctypes.c_int64, ctypes.c_int32
    lib.gdn_test_used.argtypes = [i64, i64, i32, i32, i32, i32, i32]
    lib.gdn_test_used.restype = i64
    lib.gdn_test_parts.argtypes = [i64, i64, i32, i32]
    lib.gdn_test_parts.restype = i64
    lib.nvfp4_gated_delta_workspace.argtypes = [i64] * 6 + [i32, ctypes.POINTER(i64)]
    rng, in_parts, wanted = random.Random(7), 0, i64()
    for _ in range(20000):
        k_heads = rng.choice((1, 2, 3, 8))
        sizes = (k_heads, k_heads * rng.randint(1, 6), rng.choice((64, 128)), rng.choice((64, 128, 192, 256)))
        tokens, seqs, dtype = int(2 ** rng.uniform(0, 20)), int(2 ** rng.uniform(0, 11)), rng.randint(0, 2)
        assert lib.nvfp4_gated_delta_workspace(tokens, seqs, *sizes, dtype, ctypes.byref(wanted)) == 0
        for t, n in ((tokens, seqs), (rng.randint(1, tokens), seqs), (tokens, rng.randint(1, seqs)), (tokens, 1),
                     (rng.randint(1, tokens), rng.randint(1, seqs))):
            assert lib.gdn_test_used(t, n, *sizes, dtype) <= wanted.value, (tokens, seqs, sizes, dtype, t, n)
            in_parts += lib.gdn_test_parts(t, n, sizes[1], sizes[3]) > 0
    assert in_parts > 1000


def test_convolutions_of_the_gpu_tests_reach_every_number_of_rows(tmp_path):
    """What tests/test_gpu_gdn_batches.py means to run, on a card of 256 CUs."""
    from tests.test_gpu_gdn_batches import CONV_ROWS, conv_columns

    path = str(tmp_path / "libnvfp4_gdn_rows.so")
    build(path)
    rows = ctypes.CDLL(path).gdn_test_conv_rows
    rows.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int]
    for dtype, channels, tokens, want in CONV_ROWS:
        assert rows(tokens, conv_columns(dtype, channels), channels % 8 == 0, 256) == want, (dtype, channels, tokens)
    assert {(dtype, want) for dtype, _, _, want in CONV_ROWS} == {(d, n) for d in ("f32", "bf16", "f16") for n in (8, 16, 32)}


def test_prompts_of_the_gpu_tests_are_whole_and_in_parts_as_they_mean(tmp_path):
    from tests.test_gpu_gdn_batches import BEHIND, PARTS

    path = str(tmp_path / "libnvfp4_gdn_parts.so")
    build(path)
    parts = ctypes.CDLL(path).gdn_test_parts
    parts.argtypes, parts.restype = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32], ctypes.c_int64
    for heads, lens, want in PARTS:
        assert parts(sum(lens) + BEHIND, len(lens), heads[1], heads[3]) == want, (heads, lens)
    # calls of one sequence, with what is slower: whole and in parts, both measured
    for tokens, heads, want in ((1024, 6, 0), (2048, 6, 4), (16411, 6, 21), (2048, 8, 4), (4096, 16, 8), (3000, 40, 0), (8192, 40, 6), (3000, 48, 0),
                                (4096, 48, 0), (8192, 48, 5), (8192, 56, 0), (16411, 64, 0)):
        assert parts(tokens, 1, heads, 128) == want, (tokens, heads)


def test_chunks_of_ragged_sequences_have_places_of_their_own():
    rng = random.Random(3)
    for _ in range(300):
        lens = [rng.choice((0, 0, 1, 63, 64, 65, rng.randint(0, 400))) for _ in range(rng.randint(1, 40))]
        gap = rng.randint(0, 200)
        starts = [gap]
        for n in lens:
            starts.append(starts[-1] + n)
        tokens = starts[-1] + rng.randint(0, 100)
        places = [s // 64 + r + i for r, (s, e) in enumerate(zip(starts, starts[1:])) for i in range((e - s + 63) // 64)]
        assert len(set(places)) == len(places)
        assert all(0 <= p < tokens // 64 + len(lens) for p in places)
