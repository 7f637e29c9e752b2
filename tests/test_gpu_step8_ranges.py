"""The 8-bit step and conversion where values leave the ordinary."""
import numpy as np
import pytest

import synth
from helpers import F16, F32, gen, to_dev
from test_gpu_step8 import HP, LAYOUTS, Q, make_shard, rank_buffers, real_mask

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


def decoded(sh):
    """(first moment, root of the second) as the codes and scales stand for them."""
    return [(c.float().view(-1, Q) * s.view(-1, 1)).view(-1)
            for c, s in ((sh.exp_avg8, sh.exp_avg_scale), (sh.exp_rms8, sh.exp_rms_scale))]


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


@pytest.mark.parametrize("big", [1e19, 3e20, -1e25, 1e36])
@pytest.mark.parametrize("hp", [HP, dict(HP, adamw=False, weight_decay=0.1), dict(HP, beta2=0.0)])
def test_a_finite_gradient_whose_square_overflows(big, hp):
    """The formula's root is finite, and so are the moments, this step and the next.

    Against 64 bits, u = 2^-24: the new m and r are off by 6 u of their terms' sums, the quotient by 12 u more, a
    scale by 8 u of its block's largest; a code by half an e4m3 step (2^-4, below the normal range 2^-10 scale, up to
    2^-9 scale where a root above zero takes the smallest code) and by 2^-18 for the scale's and x's own rounding."""
    at, u, shape = 5 * Q + 17, 2.0 ** -24, (-1, Q)
    sh = make_shard([Q * 40], 1, 0, 1)
    g = gen(3, synth.STREAM_GRAD, Q * 40, synth.DIST_NORMAL, 1e-3, F32).astype(np.float64)
    for step, value in ((2, big), (3, 0.5)):  # the second step's gradient is ordinary, its root is not
        g[at] = np.float32(value)
        m0, r0 = (x.cpu().numpy().astype(np.float64) for x in decoded(sh))
        w0 = sh.master.cpu().numpy().astype(np.float64)
        sh.adam_step(step=step, hyper=hp, reduced_g=to_dev(g.astype(np.float32), F32))
        b1, b2 = hp["beta1"], hp["beta2"]
        gd = g if hp["adamw"] else g + hp["weight_decay"] * w0
        m, r = b1 * m0 + (1 - b1) * gd, np.sqrt(b2 * r0 ** 2 + (1 - b2) * gd ** 2)
        a = b1 * np.abs(m0) + (1 - b1) * np.abs(gd)
        size, denom = hp["lr"] / (1 - b1 ** step), r / np.sqrt(1 - b2 ** step) + hp["eps"]
        w = w0 * (1 - hp["lr"] * hp["weight_decay"] if hp["adamw"] else 1.0) - size * m / denom
        got = sh.master.cpu().numpy().astype(np.float64)
        assert np.all(np.abs(got - w) <= 3 * u * np.abs(w0) + 20 * u * size * a / denom)
        for x, amp, back, root in zip((m, r), (a, r), decoded(sh), (False, True)):
            back = back.cpu().numpy().astype(np.float64)
            scale = np.repeat(np.abs(x).reshape(shape).max(1) / 448, Q)
            off = 8 * u * np.repeat(amp.reshape(shape).max(1) / 448, Q)
            half = np.maximum(np.abs(x) * 2.0 ** -4, (scale + off) * (2.0 ** -9 if root else 2.0 ** -10))
            assert np.all(np.abs(back - x) <= half + 2.0 ** -18 * np.abs(x) + 8 * u * amp)
            assert not root or np.all(back[x > 0] > 0)


def test_the_first_export_can_be_captured():
    sh = make_shard([100, 37, 5003], 2, 1, 64)
    dense, back = torch.zeros(sh.dense_total, device=DEV), torch.zeros_like(sh.master)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sh.to_dense(sh.master, dense)
        sh.from_dense(dense, back)
    want_dense, want_back = torch.zeros_like(dense), torch.zeros_like(back)
    sh.to_dense(sh.master, want_dense)
    sh.from_dense(want_dense, want_back)
    assert int(want_dense.count_nonzero()) > 0
    for _ in range(3):
        dense.zero_()
        back.zero_()
        torch.randn(4096, device=DEV).sum()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dense, want_dense) and torch.equal(back, want_back)


@pytest.mark.parametrize("layout", range(len(LAYOUTS)))
def test_codes_and_scales_beside_the_real_elements(layout):
    """A vector with a real element has code 0 at its padding; vectors and blocks without one are not written."""
    numels, ranks, owner, align = LAYOUTS[layout]
    sh = make_shard(numels, ranks, owner, align, moments=False)
    left = 0x39  # 1.125
    for k in ("exp_avg8", "exp_rms8"):
        getattr(sh, k).view(torch.uint8).fill_(left)
    for k in ("exp_avg_scale", "exp_rms_scale"):
        getattr(sh, k).fill_(1e-6)
    real = real_mask(sh)
    sh.adam_step(step=3, hyper=HP, rank_grads=rank_buffers(sh, 3, F16, sh.local_base), grad_base=sh.local_base,
                 divisor=3.0)
    written = np.repeat(real.reshape(-1, 8).any(1), 8)
    for k in ("exp_avg8", "exp_rms8"):
        codes = getattr(sh, k).view(torch.uint8).cpu().numpy()
        assert np.all((codes & 0x7F)[written & ~real] == 0) and np.all(codes[~written] == left), k
    touched = real.reshape(-1, Q).any(1)
    for k in ("exp_avg_scale", "exp_rms_scale"):
        scale = getattr(sh, k).cpu().numpy()
        assert np.all(scale[~touched] == np.float32(1e-6)) and np.all(scale[touched] != np.float32(1e-6)), k


@pytest.mark.parametrize("noise", [0.0, 0.3])
def test_a_fit_ends_as_with_32_bit_moments(noise):
    """The 8-bit fit's loss against the 32-bit one's, step for step the same problem.  Without noise both go
    towards 0 and the 8-bit one ends within a factor of two; with noise both end at its floor, to a thousandth."""
    torch.manual_seed(0)
    n, k = 512, 64
    x = torch.randn(n, k, device=DEV)
    y = x @ torch.randn(k, 32, device=DEV)
    y = y + noise * torch.randn(n, 32, device=DEV)
    end = {}
    for cls in (zs.OwnerShard, zs.OwnerShard8):
        sh = cls([k * 32], 1, 0, align=64, device=DEV)
        sh.alloc_state()
        for step in range(1, 301):
            e = x @ sh.master[:k * 32].view(k, 32) - y
            g = (x.t() @ e / n).reshape(-1).contiguous()
            hp = dict(HP, lr=0.05 * (1 - step / 320), beta1=0.9, beta2=0.99, weight_decay=0.0)
            sh.adam_step(step=step, hyper=hp, rank_grads=[g])
        end[cls] = float((x @ sh.master[:k * 32].view(k, 32) - y).square().mean())
    wide, narrow = end[zs.OwnerShard], end[zs.OwnerShard8]
    assert wide < 2e-3 * float(y.square().mean())
    assert narrow <= (2 * wide if noise == 0.0 else 1.001 * wide)
