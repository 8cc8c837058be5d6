"""The rotary kernels for any alignment tell the compiler no more than that: in
their intermediate code no store claims more than an element's alignment."""
import os
import re
import subprocess

import pytest

from nvfp4_w4a4_block_quantize_amd import build as b


def test_stores_claim_the_alignment_of_an_element(tmp_path):
    if not os.path.exists(b.HIPCC):
        pytest.skip("needs hipcc")
    out = str(tmp_path / "rope.ll")
    cmd = [b.HIPCC, *b.COMMON_FLAGS, "--offload-device-only", "-S", "-emit-llvm", os.path.join(b.CSRC, "rope.hip"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    kernel, seen = None, {True: 0, False: 0}
    for line in open(out):
        # rope_kernel<dtype, VEC, COPY, ADJACENT, ALIGNED, unroll>
        m = re.match(r"define .*@\w*rope_kernelILi(\d)ELi\d+ELi\d+ELb[01]ELb([01])E", line)
        if m:
            kernel = (4 if m[1] == "0" else 2, m[2] == "1")
        m = re.search(r"\bstore .*ptr addrspace\(1\).*align (\d+)", line)
        if m:
            size, aligned = kernel
            assert int(m[1]) <= (16 if aligned else size), (kernel, line)
            seen[aligned] += 1
    assert seen[True] and seen[False]
