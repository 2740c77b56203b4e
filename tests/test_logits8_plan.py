"""The kernel that dense_logits_fp8 takes for a shape (plan_logits8 of
fh_host.cpp, the function that the library asks), on the CPU: the shapes that
the GPU tests run take every kernel."""
from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

from .logits8_shapes import FAR, SHAPES, ldo

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "two_stage_retrieval_amd", "csrc")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("plan") / "logits8_plan")
    r = subprocess.run([cxx, "-std=c++17", "-O2", "-I", os.path.join(ROOT, "include"),
                        os.path.join(HERE, "host", "logits8_plan.cpp"),
                        os.path.join(CSRC, "fh_host.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def ask(shapes):
        r = subprocess.run([exe], input="\n".join(" ".join(map(str, s)) for s in shapes),
                           capture_output=True, text=True, timeout=60)
        return r.stdout.split("\n")[:-1]
    return ask


def kernels():
    """Every kernel that the library can launch, from its switches."""
    src = open(os.path.join(CSRC, "fh_logits8.hip")).read()
    tiles = {f"tiles {m} {n}" for m, n in
             re.findall(r"case \d+: enqueue_tiles<(\d+), (\d+), TO>", src)}
    rows = {f"rows {16 * int(m)} {16 * int(n)}" for m, n in
            re.findall(r"case \d+: enqueue_rows<(\d+), (\d+), TO>", src)}
    assert tiles and rows
    return tiles | rows


def test_shapes_take_the_kernels_they_are_listed_for(plan):
    for size in (2, 4):
        got = plan([(m, v, d, ldo(v, size), size) for _, m, v, d in SHAPES])
        assert got == [s[0] for s in SHAPES]
        name, m, v, d, far = FAR
        assert plan([(m, v, d, far[size], size)]) == [name]
        assert plan([(m, v, d, far[size] // 2, size)]) != [name]


def test_shapes_take_every_kernel(plan):
    assert {s[0] for s in SHAPES} == kernels()
    for name in sorted(kernels()):
        of = [s for s in SHAPES if s[0] == name]
        assert {s[3] % 128 == 0 for s in of} == {True, False}, name
        assert max(-(-s[3] // 128) for s in of) >= 3
        kind, bm, bn = name.split()
        if kind == "tiles":     # workgroups that go on to a second tile, of several blocks
            n = [-(-s[1] // int(bm)) * -(-s[2] // int(bn)) for s in of if s[3] > 256]
            assert max(n) > 256, name
            assert any(s[1] % int(bm) for s in of) and any(s[2] % int(bn) for s in of)


def test_no_shape_is_without_a_kernel(plan):
    # from one row to many, over small, odd and large vocabularies and widths
    shapes = [(m, v, d, ldo(v, size), size)
              for m in (1, 2, 4, 5, 16, 17, 31, 64, 65, 333, 2048, 65535 * 16)
              for v in (1, 15, 1000, 6144, 6145, 12288, 12289, 128256, 262144, 2 ** 28)
              for d in (16, 128, 400, 2048, 8192, 65536) for size in (2, 4)]
    got = plan(shapes)
    assert len(got) == len(shapes) and set(got) == kernels()
