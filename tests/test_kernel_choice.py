"""Which kernels the bf16 product, its gradients, the combine's gradient and the adapters
launch, on the CPU: the library's host code with a recorder in place of the runtime."""
from __future__ import annotations

import os
import subprocess

import pytest

from kernel_choices import CHOICES


@pytest.fixture(scope="module")
def record(tmp_path_factory):
    from sparse_fp4_expert_amd import build
    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not available")
    exe = build.build_launch_recorder(str(tmp_path_factory.mktemp("recorder")),
                                      ("api.cpp", "dispatch.hip", "gemm.hip", "lora.hip"))

    def run(calls):
        r = subprocess.run([exe], input="\n".join(calls) + "\n", capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stdout[-500:] + r.stderr[-500:]
        return [line.split("\t") for line in r.stdout.splitlines()]
    return run


def _name(launch):
    """A launch without its workgroups."""
    return launch.rsplit(" ", 1)[0]


def test_choices(record):
    """Every call of the table runs on its kernels, and the table leaves no kernel out: one
    that a change of the times by which they are chosen leaves without a call has
    to get one, or go."""
    wrong = []
    for (call, want), got in zip(CHOICES, record([call for call, _ in CHOICES])):
        got = got if call.startswith("lora") else [_name(g) for g in got]
        if got != want:
            wrong.append((call, want, got))
    assert not wrong, wrong
    named = {_name(k) if call.startswith("lora") else k for call, kernels in CHOICES for k in kernels}
    there = {_name(k) for k in record(["all"])[0]}
    assert there - {"permute_kernel", "unpermute_kernel", "combine_kernel"} == named


def test_columns_of_a_wave(record):
    """The table has waves of 32, 64 and 128 columns for each kernel of the second product."""
    seen = {}
    for call, kernels in CHOICES:
        if call.startswith("lora"):
            T, A, rank, slices, N, _, swiglu = (int(v) for v in call.split()[1:])
            up, groups = kernels[1].rsplit(" ", 1)
            rows = 16 * int(up.rstrip(">").split(", ")[-1])
            seg = N // max(slices, 2 if swiglu else 1)
            tiles = -(-T // rows) * (N // (2 if swiglu else 1) // seg)
            columns = [c for c in (32, 64, 128) if tiles * -(-(-(-seg // c)) // 4) == int(groups)]
            if len(columns) == 1:
                seen.setdefault(up, set()).update(columns)
    assert len(seen) == 10 and all({64, 128} <= c for c in seen.values()), seen
