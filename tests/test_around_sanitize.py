"""The argument checks of the calls around the head
(two_stage_retrieval_amd/csrc/fh_host.cpp) under the address and
undefined-behaviour sanitizers, on the CPU; tests/host/around_checks.cpp holds
the checks."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def test_workspace_of_sizes_that_are_refused():
    from two_stage_retrieval_amd import binding as fh
    size = fh.flashhead_verify_workspace_bytes
    groups = (1 << 24) - 1
    for B, rows, v in ((1, 2 ** 62, 128256), (1, 2 ** 59 + 1, 1), (1, groups + 1, 2048),
                       (1, groups // 2 + 1, 2049), (groups // 2 + 1, 1, 1),
                       (groups // 63 + 1, 1, 128256)):
        assert size(B, rows, v) == 0, (B, rows, v)
    assert size(1, groups, 2048) > groups * 16
    assert size(groups // 2, 1, 1) > groups // 2 * 16


@pytest.mark.parametrize("flags", [["-O1", "-g", "-fsanitize=address,undefined",
                                    "-fno-sanitize-recover=all"],
                                   ["-O3", "-Wall", "-Werror"]])
def test_argument_checks(tmp_path, flags):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path / "around_checks")
    r = subprocess.run([cxx, "-std=c++17", *flags, "-I", os.path.join(ROOT, "include"),
                        os.path.join(HERE, "host", "around_checks.cpp"),
                        os.path.join(ROOT, "two_stage_retrieval_amd", "csrc", "fh_host.cpp"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert int(r.stdout.split()[1]) > 500
