"""Properties of the built device code that no result shows (CPU: the library's
gfx950 code is only read)."""
from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest


def _kernels(tmp_path, *names):
    """{kernel: instructions} of the kernels with one of `names` in their symbols."""
    from sparse_fp4_expert_amd import build
    objdump = os.path.join(os.path.dirname(build.HIPCC), "..", "llvm", "bin", "llvm-objdump")
    if not os.path.exists(objdump) or not os.path.exists(build.LIB):
        pytest.skip("needs llvm-objdump and the built library")
    lib = shutil.copy(build.LIB, tmp_path)
    subprocess.run([objdump, "--offloading", lib], cwd=tmp_path, check=True, capture_output=True)
    found = {}
    for f in sorted(p for p in os.listdir(tmp_path) if p.endswith("gfx950")):
        text = subprocess.run([objdump, "-d", "--no-show-raw-insn", f], cwd=tmp_path, check=True,
                              capture_output=True, text=True).stdout
        kernel = None
        for line in text.splitlines():
            head = re.match(r"[0-9a-f]+ <(.*)>:$", line)
            if head:
                kernel = head.group(1)
            elif kernel and any(n in kernel for n in names) and line.strip():
                found.setdefault(kernel, []).append(line.split("//")[0].strip())
    return found


def test_mx_copies_carry_no_scalar_offset(tmp_path):
    """A copy to LDS behind the buffer's end has to come back as zeros.  The
    check of the range counts the lane's offset; documents differ on the
    scalar one, so the copies of the MX product have none.  (The tiled kernel
    on whole stages, its third argument true, reads nothing behind the end.)"""
    kernels = _kernels(tmp_path, "mx_stream_kernel", "mx_tiled_kernel")
    assert kernels
    for name, code in kernels.items():
        if re.search(r"mx_tiled_kernelILb[01]ELb[01]ELb1E", name):
            continue
        copies = [i for i in code if i.startswith("buffer_load") and i.split()[-1] == "lds"]
        assert copies, name
        for i in copies:
            assert re.fullmatch(r"buffer_load_dword(x4)? v\d+, s\[\d+:\d+\], 0 offen lds", i), (name, i)
