"""The bounded wait of the gated backward's dX, forced to run out from the host (GE_SK_SPIN=0 lets each
waiting workgroup poll zero times; every kernel still ends normally): each tile of dX is either the
normal one's or all NaN, gated_lost_waits counts the lost waits, and calls after it are clean. Shapes
of both protocols (test_split_lost_wait_gpu.py), eager and in a replayed graph."""
import pytest
import torch

from gemm_epilogues_epilog_amd import gated
from tests import gpu_runner as R
from tests import test_gated_gpu as G
from tests.test_split_lost_wait_gpu import tile_states

pytestmark = pytest.mark.gpu


# (m, n, k): dX is (m, k) over 2 n; a wave's part of its tile; a forced length of the runs
@pytest.mark.parametrize("m,n,k,sub,run_len", [(1024, 1024, 512, (32, 64), None), (1024, 1024, 512, (32, 64), "12"),
                                               (1024, 2048, 1024, (32, 64), None)])
def test_lost_waits(gpu, m, n, k, sub, run_len):
    x, w, _ = G.make(m, n, k, "f16", 1, bias=False)
    _, z = gated.gated_forward(x, w, save=True)
    dh = torch.randn(m, n, device="cuda").half()
    env = {"GE_SK_RUN": run_len} if run_len else {}
    run = lambda: gated.gated_backward(dh, x, w, z)   # noqa: E731
    with R.env({**env, "GE_SK_SPIN": "0"}):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            replayed = run()
    gated.gated_lost_waits()
    nans = lost = 0
    for i in range(6):
        dh.copy_(dh.roll(1, 0))
        with R.env(env):
            want = run()
            assert torch.isfinite(want.dx).all() and gated.gated_lost_waits() == 0
        if i % 2:
            replayed.dx.fill_(7.0)
            graph.replay()
            got = replayed
        else:
            with R.env({**env, "GE_SK_SPIN": "0"}):
                got = run()
        torch.cuda.synchronize()
        states = tile_states(got.dx, want.dx, *sub)
        assert "bad" not in states and torch.equal(got.dw, want.dw)
        now = gated.gated_lost_waits()
        assert 8 * now >= states.count("nan") and (now > 0) == ("nan" in states)
        nans += states.count("nan")
        lost += now
    assert gated.gated_lost_waits() == 0
    print(f"[case] {lost} waits lost, {nans} parts NaN", flush=True)


def test_null_count(gpu):
    assert gpu.load().gemm_epilog_gated_lost_waits(None, None) == 3
