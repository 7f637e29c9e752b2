"""The 8-bit step and conversion where values leave the ordinary."""
import pytest

import synth
from helpers import F32, gen, to_dev
from test_gpu_step8 import HP, Q, make_shard

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import zero_sharded_optimizer_owned_amd as zs  # noqa: E402

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    zs.lib()
    yield
    torch.cuda.synchronize()


def unpacked(sh):
    out = [torch.full_like(sh.master, -7.0) for _ in range(2)]
    sh.unpack_moments(*out)
    return out


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_both_moments_of_a_block_show_a_non_finite_gradient(bad):
    sh = make_shard([Q * 40], 1, 0, 1)
    g = to_dev(gen(3, synth.STREAM_GRAD, Q * 40, synth.DIST_NORMAL, 1e-3, F32), F32)
    g[5 * Q + 17] = bad
    sh.adam_step(step=2, hyper=HP, reduced_g=g)
    for x in unpacked(sh):
        block = torch.isnan(x).view(-1, Q)
        assert bool(block[5].all()) and int(block.any(1).sum()) == 1
        assert bool(torch.isfinite(x.view(-1, Q)[[i for i in range(40) if i != 5]]).all())


@pytest.mark.parametrize("bad", [float("inf"), float("nan"), -1.0])
def test_packing_a_second_moment_that_is_no_number(bad):
    """An infinite or negative exp_avg_sq makes its block's roots NaN, the first moment and other blocks hold."""
    sh = zs.OwnerShard8([Q * 3], 1, 0, align=1, device=DEV)
    sh.alloc_state()
    m, v = torch.full((Q * 3,), 0.5, device=DEV), torch.full((Q * 3,), 0.25, device=DEV)
    v[Q + 1] = bad
    sh.pack_moments(m, v)
    gm, gv = unpacked(sh)
    assert bool((gm == 0.5).all())
    assert bool(torch.isnan(gv[Q:2 * Q]).all()) and bool(torch.isfinite(gv[:Q]).all() and torch.isfinite(gv[2 * Q:]).all())
