"""The root-mean-square norm, its 8-bit form and its backward pass against their
definitions in 64 bits.

Tolerances.  u = 2^-24.  rstd is formed in fp64 and rounded once: u relative.
out = h rstd gain: rstd and two products, 3 u, and the store's half step.  The
codes and scales are whole steps of given fp32 operations, 448 (1 / max) and
max (1 / 448): equal bit for bit.  n carries 2 u (3 u from the kept form), d one;
a mean of D products carries 10 u of their mean magnitude (chains of 8 in fp32,
the rest in fp64), so
  dx is off by u rstd (8 |d| + 8 |n m|) + 14 u rstd |n| mean|d n| + 2 u |dx|,
  dgain by (L + 6) u sum|dy n|, L the longest fp32 chain of one block's rows,
and each by its store's half step.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import zero_sharded_optimizer_owned_amd as zs  # noqa: E402

DEV = "cuda"
U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SUB = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}
SHAPES = [(1, 1), (1, 8), (3, 7), (5, 128), (2, 129), (4, 255), (7, 512), (6, 513), (9, 1000), (5, 1024), (3, 1025),
          (4, 2047), (5, 4096), (3, 4099), (2, 5003), (3, 8192), (2, 8200), (2, 16_384), (2, 16_383), (1500, 40), (2100, 300)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    zs.lib()
    yield
    torch.cuda.synchronize()


def within(got, want, tol):
    got, want, tol = got.double().cpu(), want.cpu(), tol.cpu()
    off = (got - want).abs() - tol
    assert not torch.isnan(got).any() and float(off.max()) <= 0, (float(off.max()), int(off.argmax()))


def half_step(x, dt):
    return x.abs() * (torch.finfo(DT[dt]).eps / 2) + SUB[dt]


def rows(n, d, dt, seed, spread=1.0):
    """At an odd address: rows need no alignment."""
    g = torch.Generator().manual_seed(seed + 13 * n + d)
    x = torch.randn(n, d, generator=g) * spread
    if d > 20:
        x[:, d // 3] *= 30  # one channel far larger than the rest
    buf = torch.empty(n * d + 3, dtype=DT[dt], device=DEV)
    buf[1:1 + n * d].copy_(x.reshape(-1))
    return buf[1:1 + n * d].view(n, d)


def kept_reference(h):
    """Codes as fp32 values and scales, by the same fp32 operations on the host."""
    h = h.float().cpu()
    n, d = h.shape
    blocks = -(-d // 128)
    b = torch.nn.functional.pad(h, (0, blocks * 128 - d)).view(n, blocks, 128)
    top = b.abs().amax(2, keepdim=True)
    live = top >= 2.0 ** -100
    one = torch.ones((), dtype=torch.float32)
    inv = torch.where(live, 448 * (one / top), 0 * one)
    codes = (b * inv).to(torch.float8_e4m3fn).float().view(n, -1)[:, :d]
    return codes, torch.where(live, top * (one / 448), 0 * one)[:, :, 0]


def forward(x, gain, residual=None, keep=False, eps=1e-6):
    n, d = x.shape
    h = torch.full_like(x, 7.0) if residual is not None else None
    out, rstd = torch.full_like(x, 7.0), torch.empty(n, device=DEV)
    codes = torch.empty(n, d, dtype=torch.float8_e4m3fn, device=DEV) if keep else None
    scales = torch.empty(n, -(-d // 128), device=DEV) if keep else None
    zs.zero_rms_norm(x, gain, out, residual=residual, h=h, eps=eps, rstd=rstd, codes=codes, scales=scales)
    return h if h is not None else x, out, rstd, codes, scales


@pytest.mark.parametrize("keep, residual", [(False, False), (True, True), (False, True)])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("n, d", SHAPES)
def test_forward(n, d, dt, keep, residual):
    x, gain = rows(n, d, dt, 1), rows(1, d, dt, 2)[0].contiguous()
    res = rows(n, d, dt, 3, 4.0) if residual else None
    h, out, rstd, codes, scales = forward(x, gain, res, keep)
    if residual:
        assert torch.equal(h.cpu(), (x.cpu().float() + res.cpu().float()).to(DT[dt]))
    e = h.double().cpu()
    want = (e.pow(2).mean(1) + 1e-6) ** -0.5
    within(rstd, want, 1.001 * U * want)
    y = e * want[:, None] * gain.double().cpu()
    within(out, y, 3.01 * U * y.abs() + half_step(y, dt))
    if keep:
        c, s = kept_reference(h)
        assert torch.equal(codes.float().cpu(), c) and torch.equal(scales.cpu(), s)


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("upstream", [False, True])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("n, d", SHAPES)
def test_backward(n, d, dt, keep, upstream):
    x, gain, dy = rows(n, d, dt, 1), rows(1, d, dt, 2)[0].contiguous(), rows(n, d, dt, 4, 0.5)
    _, _, rstd, codes, scales = forward(x, gain, keep=True)
    up = rows(n, d, dt, 5) if upstream else None
    dx, dgain = torch.full_like(dy, 7.0), torch.full_like(gain, 7.0)
    ws = zs.rms_norm_workspace(n, d)
    ws.fill_(0xA5)
    held = dict(codes=codes, scales=scales) if keep else dict(h=x)
    zs.zero_rms_norm_backward(dy, gain, rstd, dx, dgain, workspace=ws, upstream=up, **held)
    r, g, e = rstd.double().cpu()[:, None], gain.double().cpu(), dy.double().cpu()
    s = scales.double().cpu().repeat_interleave(128, 1)[:, :d]
    norm = (codes.double().cpu() * s if keep else x.double().cpu()) * r
    dn = e * g
    m = (dn * norm).mean(1, keepdim=True)
    want = r * (dn - norm * m) + (0 if up is None else up.double().cpu())
    size = (dn * norm).abs().mean(1, keepdim=True)
    tol = U * (r * (8 * dn.abs() + 8 * (norm * m).abs()) + 14 * r * norm.abs() * size + 2 * want.abs())
    within(dx, want, tol + half_step(want, dt))
    chain = n // 512 + 12
    want, size = (e * norm).sum(0), (e * norm).abs().sum(0)
    within(dgain, want, (chain + 6) * U * size + half_step(want, dt))
    # in place of dy and of the upstream gradient: the same bits
    for into in ("dy", "up"):
        if into == "up" and up is None:
            continue
        a, b = dy.clone(), None if up is None else up.clone()
        again = torch.empty_like(dgain)
        zs.zero_rms_norm_backward(a, gain, rstd, a if into == "dy" else b, again, workspace=ws, upstream=b, **held)
        assert torch.equal(a if into == "dy" else b, dx) and torch.equal(again, dgain)


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("n, d", SHAPES)
def test_restore(n, d, dt):
    x, gain = rows(n, d, dt, 1), rows(1, d, dt, 2)[0].contiguous()
    _, _, rstd, codes, scales = forward(x, gain, keep=True)
    out = torch.full_like(x, 7.0)
    zs.zero_rms_norm_restore(codes, scales, rstd, gain, out)
    s = scales.double().cpu().repeat_interleave(128, 1)[:, :d]
    want = codes.double().cpu() * s * rstd.double().cpu()[:, None] * gain.double().cpu()
    within(out, want, 3.01 * U * want.abs() + half_step(want, dt))


def test_gradient_against_differences():
    """dx and dgain along random directions against the change of sum(out * w) in 64 bits."""
    n, d = 6, 200
    x, gain, w = rows(n, d, "f32", 1), rows(1, d, "f32", 2)[0].contiguous(), rows(n, d, "f32", 3)
    _, _, rstd, _, _ = forward(x, gain)
    dx, dgain = torch.empty_like(x), torch.empty_like(gain)
    zs.zero_rms_norm_backward(w, gain, rstd, dx, dgain, workspace=zs.rms_norm_workspace(n, d), h=x)
    xd, gd, wd = x.double().cpu(), gain.double().cpu(), w.double().cpu()

    def value(a, b):
        return (a * (a.pow(2).mean(1, keepdim=True) + 1e-6) ** -0.5 * b * wd).sum()

    gen = torch.Generator().manual_seed(9)
    for _ in range(5):
        p, q = torch.randn(n, d, generator=gen, dtype=torch.float64), torch.randn(d, generator=gen, dtype=torch.float64)
        t = 1e-5
        slope = (value(xd + t * p, gd + t * q) - value(xd - t * p, gd - t * q)) / (2 * t)
        got = (dx.double().cpu() * p).sum() + (dgain.double().cpu() * q).sum()
        size = (dx.double().cpu() * p).abs().sum() + (dgain.double().cpu() * q).abs().sum()
        # the gradients' own 30 u, and the third derivative's share of the difference, some t^2 of the size
        assert abs(got - slope) <= 60 * U * size + 1e-8 * size


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_zeros_large_and_non_finite_rows(dt):
    d = 300
    x = rows(8, d, dt, 1)
    x[1] = 0
    x[2] = 3e38  # squares past fp32
    x[3] = 1e-36
    x[4, 7], x[5, 260] = float("inf"), float("nan")
    x[6, :128] = 0  # one block of zeros
    gain = torch.ones(d, dtype=DT[dt], device=DEV)
    _, out, rstd, codes, scales = forward(x, gain, keep=True)
    assert (out[1] == 0).all() and (codes[1].float() == 0).all() and (scales[1] == 0).all()
    assert torch.allclose(out[2].float(), torch.ones(d, device=DEV), rtol=2 ** -7)
    # a row far below eps: out = x / sqrt(eps); its codes are zeros (its maximum is below 2^-100)
    want = x[3].double() * 1e3
    assert ((out[3].double() - want).abs() <= 2.0 ** -7 * want.abs() + 1e-40).all()
    assert (codes[3].float() == 0).all() and (scales[3] == 0).all()
    assert torch.isnan(scales[4, 0]) and not torch.isnan(scales[4, 1:]).any()  # its own block only
    assert torch.isnan(scales[5, 2]) and not torch.isnan(scales[5, :2]).any()
    assert torch.isnan(out[5]).all() and torch.isnan(rstd[5])
    assert (codes[6, :128].float() == 0).all() and scales[6, 0] == 0 and scales[6, 1] > 0
    for i in (0, 7):
        assert torch.isfinite(out[i].float()).all()


def test_in_place_and_no_rows():
    n, d = 5, 777
    x, res, gain = rows(n, d, "bf16", 1), rows(n, d, "bf16", 2), rows(1, d, "bf16", 3)[0].contiguous()
    h, out, _, _, _ = forward(x, gain, res)
    a, b = x.clone(), res.clone()
    zs.zero_rms_norm(a, gain, a, residual=b, h=b)  # h over the residual, out over x
    assert torch.equal(a, out) and torch.equal(b, h)
    none, dgain = torch.empty(0, d, dtype=torch.bfloat16, device=DEV), torch.full_like(gain, 7.0)
    zs.zero_rms_norm(none, gain, none)
    zs.zero_rms_norm_backward(none, gain, torch.empty(0, device=DEV), none, dgain, workspace=zs.rms_norm_workspace(0, d), h=none)
    assert (dgain == 0).all()


def test_more_rows_than_blocks_is_the_same_every_time():
    n, d = 9000, 96
    x, gain, dy = rows(n, d, "f32", 1), rows(1, d, "f32", 2)[0].contiguous(), rows(n, d, "f32", 4)
    _, _, rstd, _, _ = forward(x, gain)
    ws, seen = zs.rms_norm_workspace(n, d), None
    for _ in range(3):
        dx, dgain = torch.empty_like(x), torch.empty_like(gain)
        zs.zero_rms_norm_backward(dy, gain, rstd, dx, dgain, workspace=ws, h=x)
        assert seen is None or (torch.equal(seen[0], dx) and torch.equal(seen[1], dgain))
        seen = dx, dgain
    e = (dy.double() * x.double() * rstd.double()[:, None]).cpu()
    within(seen[1], e.sum(0), (n // 512 + 18) * U * e.abs().sum(0))


def test_binding_refuses():
    x, g = torch.zeros(3, 16, device=DEV), torch.zeros(16, device=DEV)
    r, ws = torch.zeros(3, device=DEV), zs.rms_norm_workspace(3, 16)
    c, s = torch.zeros(3, 16, dtype=torch.float8_e4m3fn, device=DEV), torch.zeros(3, 1, device=DEV)
    for bad in (dict(x=x[:, ::2]), dict(gain=g[:8]), dict(gain=g.half()), dict(out=x[:2]), dict(residual=x), dict(h=x),
                dict(codes=c), dict(codes=c, scales=s[:2]), dict(codes=c.view(torch.uint8), scales=s), dict(rstd=r[:2]),
                dict(x=x.double())):
        with pytest.raises((ValueError, TypeError)):
            zs.zero_rms_norm(**{**dict(x=x, gain=g, out=x.clone()), **bad})
    good = dict(dy=x, gain=g, rstd=r, dx=x.clone(), dgain=g.clone(), workspace=ws)
    for bad in (dict(), dict(h=x, codes=c, scales=s), dict(codes=c), dict(h=x[:2]), dict(h=x, upstream=x.half()),
                dict(h=x, dgain=g[:3])):
        with pytest.raises((ValueError, TypeError)):
            zs.zero_rms_norm_backward(**{**good, **bad})
    with pytest.raises(zs.ZeroShardError):
        zs.zero_rms_norm_backward(**{**good, "h": x, "workspace": ws[:64]})
    big = torch.zeros(1, 20_000, device=DEV)
    with pytest.raises(zs.ZeroShardError):
        zs.zero_rms_norm(big, big[0], big)
