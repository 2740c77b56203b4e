"""The largest calls of dense_logits_int4: a launch has 2^32 threads along a
dimension less one at most, and a call that would need more is refused."""
from __future__ import annotations

import os
import random
import re
import shutil
import subprocess

import pytest

from .logits4_shapes import SHAPES

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "two_stage_retrieval_amd", "csrc")
OK, UNSUPPORTED = 0, -3


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ not available")
    exe = str(tmp_path_factory.mktemp("grid") / "logits4_grid")
    r = subprocess.run([cxx, "-std=c++17", "-O2", "-I", os.path.join(ROOT, "include"),
                        os.path.join(HERE, "host", "logits4_grid.cpp"),
                        os.path.join(CSRC, "fh_host.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(shapes):
        r = subprocess.run([exe], input="\n".join(" ".join(map(str, s)) for s in shapes),
                           capture_output=True, text=True, timeout=60)
        out = [line.split() for line in r.stdout.split("\n")[:-1]]
        assert len(out) == len(shapes)
        return [(name, int(threads), int(status)) for name, threads, status in out]
    return run


def launched(name, rows, v):
    """The threads by the source of the kernels: their template arguments."""
    src = open(os.path.join(CSRC, "fh_int4.hip")).read()
    kind, args = re.search(r"case Logits4Plan::%s:\s*(?:if constexpr \(!?kF32\))?\s*"
                           r"enqueue_(rows|tiles)<([^>]*)>" % name, src).groups()
    m, n, w = (int(x) for x in args.split(",")[:3])
    if kind == "rows":
        return -(-v // (16 * n)) * 64 * w
    return 8 * -(-(-(-v // (16 * n * w))) // 8) * -(-rows // (16 * m)) * 64 * w


def test_status_codes():
    header = open(os.path.join(ROOT, "include", "flashhead.h")).read()
    value = dict(re.findall(r"(FH_OK|FH_ERR_UNSUPPORTED)\s*=?\s*\(?(-?\d+)", header))
    assert {k: int(x) for k, x in value.items()} == {"FH_OK": OK, "FH_ERR_UNSUPPORTED": UNSUPPORTED}


def test_threads_are_those_of_the_launch(ask):
    rng = random.Random(1)
    some = [(rows, v, int(h == "f32")) for h in SHAPES for _, rows, v, _ in SHAPES[h]]
    some += [(int(2 ** rng.uniform(0, 20)), int(2 ** rng.uniform(0, 28)), rng.randrange(2))
             for _ in range(3000)]
    got = ask(some)
    assert len({name for name, _, _ in got}) == 8
    for (rows, v, _), (name, threads, status) in zip(some, got):
        assert threads == launched(name, rows, v)
        assert status != OK or threads < 1 << 32, (rows, v, name)
        fits = rows <= 65535 * 16 and rows * -(-v // 256) <= 1 << 29 and threads < 1 << 32
        assert status == (OK if fits else UNSUPPORTED), (rows, v, name)


def test_calls_at_the_limit(ask):
    """ceil(rows / 64) * ceil(v / 2048) below 2^20 for an fp32 h."""
    calls = [(262144, 2048 * 256, 1), (1046526, 513 * 256, 1), (262080, 2048 * 256, 1),
             (262144, 2040 * 256, 1), (262144, 2041 * 256, 1), (262144, 2048 * 256, 0),
             (65535 * 16, 512 * 256, 1), (65535 * 16 - 64, 512 * 256, 1)]
    got = ask(calls)
    for (rows, v, f32), (name, _, status) in zip(calls, got):
        assert name == ("k64x256" if f32 else "k64x512")
        fits = not f32 or -(-rows // 64) * -(-v // 2048) < 1 << 20
        assert status == (OK if fits else UNSUPPORTED), (rows, v, f32)
    assert [status for _, _, status in got].count(OK) == 4
