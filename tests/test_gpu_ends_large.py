"""The embedding, norm and linear cross entropy calls on arrays past 2^32 bytes or elements.

What small arrays are tested for is not repeated: rows at the far end are compared with a
call on them alone, sums with whole numbers, the linear cross entropy with its definition in
64 bits at the tolerances of test_gpu_head.py, at rows and columns of both ends.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import zero_sharded_optimizer_owned_amd as zs  # noqa: E402

DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    zs.lib()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def test_norm_of_more_than_2_32_elements():
    n, d = 270_000, 16_384
    assert n * d > 2 ** 32
    g = torch.Generator(DEV).manual_seed(1)
    x = torch.empty(n, d, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    gain = torch.empty(d, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    out, rstd = torch.empty_like(x), torch.empty(n, device=DEV)
    codes = torch.empty(n, d, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty(n, d // 128, device=DEV)
    zs.zero_rms_norm(x, gain, out, rstd=rstd, codes=codes, scales=scales)
    few = slice(n - 7, n)
    part = [torch.empty_like(t[few]) for t in (out, rstd, codes, scales)]
    zs.zero_rms_norm(x[few], gain, part[0], rstd=part[1], codes=part[2], scales=part[3])
    for whole, alone in zip((out, rstd, codes, scales), part):
        assert torch.equal(whole[few].float(), alone.float())
    # backward from either form, dx over dy; dgain is off by its chains and its half step
    dgain, one = torch.empty_like(gain), torch.empty_like(gain)
    dy = out  # any values
    for held in (dict(h=x), dict(codes=codes, scales=scales)):
        want, size = (torch.zeros(d, dtype=torch.float64, device=DEV) for _ in range(2))
        for r0 in range(0, n, 2000):
            r = slice(r0, r0 + 2000)
            e = x[r].double() if "h" in held else codes[r].double() * scales[r].double().repeat_interleave(128, 1)
            e *= rstd[r].double()[:, None] * dy[r].double()
            want += e.sum(0)
            size += e.abs().sum(0)
        dx = torch.empty_like(part[0])
        zs.zero_rms_norm_backward(dy[few].contiguous(), gain, rstd[few], dx, one, workspace=zs.rms_norm_workspace(7, d),
                                  **{k: t[few] for k, t in held.items()})
        zs.zero_rms_norm_backward(dy, gain, rstd, dy, dgain, workspace=zs.rms_norm_workspace(n, d), **held)
        assert torch.equal(dy[few], dx)
        assert ((dgain.double() - want).abs() <= (n / 512 + 18) * U * size + 2.0 ** -8 * want.abs()).all()
    zs.zero_rms_norm_restore(codes, scales, rstd, gain, out)
    zs.zero_rms_norm_restore(codes[few], scales[few], rstd[few], gain, part[0])
    assert torch.equal(out[few], part[0])


def test_embedding_of_more_than_2_32_elements():
    n, v, d = 2_200_000, 50, 2048
    assert n * d > 2 ** 32
    table = torch.randn(v, d, device=DEV).bfloat16()
    tokens = torch.arange(n, device=DEV) % (v + 1)  # the last one lies outside the table
    out = torch.empty(n, d, dtype=torch.bfloat16, device=DEV)
    zs.zero_embedding(table, tokens, out)
    for at in (slice(0, 500), slice(n - 500, n)):
        ok = tokens[at] < v
        assert torch.equal(out[at][ok], table[tokens[at][ok]]) and (out[at][~ok] == 0).all()
    out.fill_(1.0)
    out[n - 100:] = 2.0
    dtable = torch.empty(v, d, device=DEV)
    zs.zero_embedding_grad(out, tokens, dtable, workspace=zs.embedding_workspace(n, v, d))
    count = torch.bincount(tokens, minlength=v + 1) + torch.bincount(tokens[n - 100:], minlength=v + 1)
    assert (dtable == count[:v, None].float()).all()


def bounds(h, w, lp, at, x, weight, divisor, eps):
    """softmax - onehot times its factor, and how far off it may be."""
    d = h.shape[1]
    e = (2 * (d / 32 + 8) * U * (h.abs() @ w.abs().T)).max(1).values
    z = (x.max(1).values - x.min(1).values).clamp(max=42)
    row = torch.arange(len(at), device=DEV)
    r = 2 * e + (6 * torch.maximum(z, -lp[row, at]) + 40) * U
    coef = weight / divisor
    dx = coef[:, None] * lp.exp()
    dx[row, at] = coef * torch.expm1(lp[row, at])
    off = (r[:, None] + 1.01 * 2.0 ** -11 + eps / 2) * dx.abs() + 2.0 ** -38 * coef.abs().max()
    off[row, at] = (r + eps / 256) * dx[row, at].abs() + 2.0 ** -38 * coef.abs().max()
    return dx, off, r


def near(got, want, off, mags, k, eps):
    tol = off + 2 * (k / 32 + 70) * U * mags
    tol = tol + (eps / 2) * (want.abs() + tol) + 2.0 ** -134
    by = (got.double() - want).abs() - tol
    assert not torch.isnan(by).any() and float(by.max()) <= 0, float(by.max())


@pytest.mark.parametrize("n, v, d", [(16_384, 200_000, 8), (20, 1 << 20, 2304), (3, 1 << 20, 2304)])
def test_linear_cross_entropy_past_2_32_bytes(n, v, d):
    """16,384 rows of 200,000 logits at once (6.6 GB), and weights of 4.8 GB."""
    assert max(n * v, v * d) * 2 > 2 ** 32
    g = torch.Generator(DEV).manual_seed(n)
    h = torch.empty(n, d, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    w = torch.empty(v, d, dtype=torch.bfloat16, device=DEV).normal_(0, 2 / math.sqrt(d), generator=g)
    t = torch.randint(0, v, (n,), generator=g, device=DEV)
    t[0], t[n - 1] = v - 1, v - 2
    weight = torch.rand(n, generator=g, device=DEV) + 0.1
    stats, logp, dh, dw = torch.empty(2, device=DEV), torch.empty(n, device=DEV), torch.empty_like(h), torch.empty_like(w)
    zs.zero_linear_cross_entropy(h, w, t, row_weight=weight, divisor=3.0, stats=stats, logp=logp, dhidden=dh, dweight=dw,
                                 workspace=zs.linear_cross_entropy_workspace(n, v, d, piece_rows=16_384), piece_rows=16_384)
    eps, wd = 2.0 ** -7, w.double()
    columns = torch.cat([torch.arange(300, device=DEV), torch.arange(v - 300, v, device=DEV)])
    want_w, off_w, mag_w = (torch.zeros(len(columns), d, dtype=torch.float64, device=DEV) for _ in range(3))
    loss = size = 0.0
    for r0 in range(0, n, 1024):
        rows = slice(r0, min(n, r0 + 1024))
        hd, at = h[rows].double(), t[rows]
        x = hd @ wd.T
        lp = torch.log_softmax(x, 1)
        row = torch.arange(len(at), device=DEV)
        dx, off, r = bounds(hd, wd, lp, at, x, weight[rows].double(), 3.0, eps)
        said = lp[row, at]
        assert ((logp[rows].double() - said).abs() <= r + U * said.abs()).all()
        loss += float(-(weight[rows].double() / 3.0 * said).sum())
        size += float((weight[rows].double() / 3.0 * (r + U * said.abs())).sum())
        if r0 == 0 or rows.stop == n:
            near(dh[rows], dx @ wd, off @ wd.abs(), dx.abs() @ wd.abs(), v, eps)
        want_w += dx[:, columns].T @ hd
        off_w += off[:, columns].T @ hd.abs()
        mag_w += dx[:, columns].abs().T @ hd.abs()
        del x, lp, dx, off
    near(dw[columns], want_w, off_w, mag_w, n, eps)
    assert abs(float(stats[0]) - loss) <= size + 2 * U * abs(loss) and int(stats[1]) == n
