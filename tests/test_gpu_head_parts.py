"""Linear cross entropy where dhidden's sums are cut into parts of the vocabulary, and at
the sizes past which its kernels go round again, against the definition in 64 bits.

The tolerances are those of test_gpu_head.py: a sum cut into s parts adds s - 1 terms
to the K / 32 of its products, which the 70 of their bound hold (s is at most 64).
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import zero_sharded_optimizer_owned_amd as zs  # noqa: E402
from test_gpu_head import check, problem, run  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    zs.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("n, v, d, piece", [
    (300, 5001, 264, 8192),   # one tile of 256 rows, two of columns, 9 parts
    (700, 3000, 264, 8192),   # three by two, 5 parts
    (1500, 9000, 520, 8192),  # five by three, 16 parts
    (700, 5001, 72, 300),     # three pieces of two, two and one tile
    (1300, 4000, 40, 512),    # the last piece smaller
    (400, 20_000, 8, 8192),   # many parts of few columns
])
def test_dhidden_in_parts(n, v, d, piece, dt):
    h, w, t, weight = problem(n, v, d, dt)
    scale = 1024.0 if dt == "f16" else 1.0
    got = run(h, w, t, weight, grad_scale=scale, piece=piece)
    check(h, w, t, weight, got, dt, grad_scale=scale)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_rows_of_more_tiles_than_one_round_of_the_softmax(dt):
    """More than 512 tiles of 256 columns to a row, which one block goes over."""
    n, v, d = 520, 131_500, 16
    h, w, t, weight = problem(n, v, d, dt)
    got = run(h, w, t, weight)
    check(h, w, t, weight, got, dt)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("n, v", [(5300, 256), (6000, 200), (9500, 300)])
def test_more_targets_in_one_tile_than_its_list_holds(n, v, dt):
    """More than 4096 rows that count have their target in one tile of dweight's product."""
    h, w, t, weight = problem(n, v, 8, dt)
    t[t == v - 1] = 3
    assert int(((t >= 0) & (t < min(v, 256))).sum()) > 4096
    got = run(h, w, t, weight, piece=16_384)
    check(h, w, t, weight, got, dt)


def test_a_larger_workspace_s_first_result_is_the_definition_s():
    """The shape that other tests compare with itself only."""
    h, w, t, weight = problem(700, 3000, 264, "bf16")
    ws = zs.linear_cross_entropy_workspace(1000, 3000, 264)
    check(h, w, t, weight, run(h, w, t, weight, ws=ws), "bf16")
