"""The shapes of gated_shapes.py reach the kernels that they are there for: the host rules built with
g++ and asked (tests/sanitize/gated_routes.cpp)."""
import os
import shutil
import subprocess

import pytest

from tests import gated_shapes as S

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "gemm_epilogues_epilog_amd", "csrc")


@pytest.fixture(scope="module")
def routes(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path_factory.mktemp("routes") / "routes")
    cmd = ["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           *(os.path.join(CSRC, f) for f in ("gated_host.cpp", "w4_host.cpp", "plan_host.cpp")),
           os.path.join(HERE, "sanitize", "gated_routes.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]

    def ask(*lines):
        r = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, lines
        return r.stdout.splitlines()
    return ask


def line(op, *sizes):
    return " ".join([op, *(str(int(v)) for v in sizes)])


def test_forward(routes):
    assert routes(*(line("forward", *s) for s in S.FORWARD)) == list(S.FORWARD.values())


def test_down(routes):
    assert routes(*(line("down", *s) for s in S.DOWN)) == list(S.DOWN.values())


def test_backward(routes):
    for (m, n, k, d, t), want in S.BACKWARD.items():
        got = routes(line("gradient", m, n, d, t), line("product", m, k, 2 * n, t, 0), line("product", 2 * n, k, m, t, 1),
                     line("product", d, n, m, t, 1))
        assert tuple(got) == want, (m, n, k, d, t)


def test_w4(routes):
    got = routes(*(line("w4", m, n, k, group, gated, k % 8 == 0) for m, n, k, group, gated in S.W4))
    assert got == list(S.W4.values())
