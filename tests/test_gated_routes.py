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


def test_lanes_of_a_launch(routes):
    """A launch has fewer than 2^32 lanes, whichever kernel takes its rows."""
    cdiv = lambda a, b: -(-a // b)   # noqa: E731
    for n in (1, 7, 8, 32, 33, 64, 65, 100, 2752, 11008, 1 << 20):
        for gated in (0, 1):
            rows = int(routes(line("rows", n, gated))[0])
            assert rows >= 256 and rows % 256 == 0
            # tiles and lanes of the general kernel and of the tile kernels (gated: half their columns)
            for bm, bn, lanes in ((64, 64, 256), (128, 128, 256), (128, 128, 512), (128, 256, 512), (192, 256, 512), (256, 256, 512)):
                assert cdiv(rows, bm) * cdiv(n, bn // (1 + gated)) * lanes < 1 << 32, (n, gated, bm, bn)
            for tile, (bm, bn) in enumerate(((256, 256), (192, 256), (128, 128), (64, 128))):
                rows = int(routes(line("w4rows", n, gated, tile))[0])
                assert rows >= bm and rows % bm == 0 and rows // bm * cdiv(n * (1 + gated), bn) * 512 < 1 << 32


def test_room_for_the_column_sums(routes):
    for m in (1, 7, 32, 33, 77, 128, 129, 2048, 2049, 16384, 100000, 1 << 24):
        for n in (1, 7, 8, 264, 1101, 4096, 11008, 1 << 20):
            for d in (8, 33, 4096):
                for t in (S.F32, S.F16, S.BF16):
                    most, used, room = map(int, routes(line("sums", m, n, 8, d, t))[0].split())
                    assert 1 <= most <= used <= room, (m, n, d, t)


@pytest.mark.parametrize("tile", ["S", "M", "L", "LH", "LM", "LM4", "LMD", "L3", "LW"])
def test_a_forced_tile(routes, monkeypatch, tile):
    """GE_TILE, for experiments with plans, also names tiles that the gated products do not have: the rules
    then choose one that they do have, as its grid is made for it."""
    monkeypatch.setenv("GE_TILE", tile)
    kernels = {"L", "L3", "LW", "LM", "LMD"}
    for m, n, k in ((77, 1000, 520), (512, 4096, 2048), (2048, 2048, 256), (4096, 11008, 4096)):
        forward, gradient = (r.split()[0] for r in routes(line("forward", m, n, k, S.BF16), line("gradient", m, n, k, S.BF16)))
        assert gradient in kernels and forward in kernels - {"L3", "LW"} | {"few"}
        if tile in kernels:
            assert gradient == tile
