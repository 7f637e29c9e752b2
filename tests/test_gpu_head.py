"""Linear cross entropy against its definition in 64 bits.

Tolerances.  u = 2^-24.  A logit is a product of D terms added in fp32 by 32 at
a time, truncation allowed for: off by at most e = 2 (D / 32 + 8) u sum|h w| / T.
With E the row's largest e and z = max |x - x_max| over logits that matter
(exp(-z) above 2^-60),
  lp is off by 2 E + (6 z + 40) u + u |lp| (each term of the row's sum carries its
  own e, 2.5 u z and a few u), and
  softmax - onehot by r = 2 E + (6 z + 40) u relative.
What is held of it is rounded to 11 bits within its 256 columns and once more to
the storage type, relative to the largest weight and down to 2^-38 of it:
  |d dx| <= (r + 1.01 2^-11 + eps / 2) |dx| + 2^-38 c,  c = grad_scale max|w| / (divisor T),
and at the target, whose residual is kept, by r + 2^-8 eps (itself in 16 bits, or fp32).
(A number m 2^k with 11 significant bits, 1 <= m < 2, lies on a grid of step
2^(k - 10): rounding to it is off by at most 2^(k - 11), so 2^-11 of the number, as
eps / 2 is for fp16 and 2^-8 for bf16; the 1.01 holds the product of the two.)
The products then add K terms in fp32 (2 (K / 32 + 70) u of their magnitudes) and
round to the storage type.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import zero_sharded_optimizer_owned_amd as zs  # noqa: E402

DEV = "cuda"
U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
SUB = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}
#         rows, vocab, dim, piece rows
SHAPES = [(1, 1, 8, 8192), (1, 2, 8, 8192), (1, 1000, 64, 8192), (2, 15, 72, 8192), (5, 17, 16, 8192), (16, 4097, 136, 8192),
          (17, 257, 40, 8192), (33, 1000, 200, 8192), (77, 5001, 328, 8192), (255, 256, 64, 8192), (256, 512, 128, 8192),
          (257, 300, 264, 8192), (600, 2047, 96, 8192), (1025, 700, 512, 8192), (300, 1030, 520, 128), (50, 999, 80, 16),
          (40, 333, 56, 7), (513, 129, 1032, 256), (8, 600, 136, 8192), (9, 600, 136, 8192), (128, 800, 72, 8192),
          (129, 800, 72, 8192), (400, 40, 264, 8192), (3000, 60, 24, 8192)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    zs.lib()
    yield
    torch.cuda.synchronize()


def matrix(n, d, dt, g, spread, pad):
    """[n, d] at a row stride with other values between the rows, and the buffer."""
    buf = torch.full((max(1, n) * (d + pad) + 8,), 3.0, dtype=DT[dt], device=DEV)
    t = buf[8:8 + n * (d + pad)].view(n, d + pad)[:, :d]
    t.copy_(torch.randn(n, d, generator=g) * spread)
    return t, buf


def problem(n, v, d, dt, seed=0, spread=2.0, pad=0, ignore=0.2):
    g = torch.Generator().manual_seed(seed + n + 3 * v + 5 * d)
    h, _ = matrix(n, d, dt, g, 1.0, pad)
    w, _ = matrix(v, d, dt, g, spread / math.sqrt(d), pad)
    t = torch.randint(0, v, (n,), generator=g)
    if n > 2:
        t[torch.rand(n, generator=g) < ignore] = -100
        t[0] = v - 1
        t[1] = v  # outside as well
    weight = (torch.rand(n, generator=g) + 0.1).to(DEV)
    return h, w, t.to(DEV), weight


def run(h, w, t, weight, divisor=3.0, temperature=1.0, grad_scale=1.0, grads=(True, True), piece=8192, ws=None, pad=0, **out):
    n, d = h.shape
    v = w.shape[0]
    stats, logp = torch.full((2,), 9.0, device=DEV), torch.full((n,), 9.0, device=DEV)
    make = lambda m: torch.full((m, d + pad), 5.0, dtype=h.dtype, device=DEV)[:, :d]  # noqa: E731
    dh, dw = make(n) if grads[0] else None, make(v) if grads[1] else None
    if ws is None:
        ws = zs.linear_cross_entropy_workspace(n, v, d, grad=any(grads), piece_rows=piece)
        ws.fill_(0xA5)
    zs.zero_linear_cross_entropy(h, w, t, row_weight=weight, divisor=divisor, temperature=temperature, grad_scale=grad_scale,
                                 stats=stats, logp=logp, dhidden=dh, dweight=dw, workspace=ws, piece_rows=piece)
    return stats, logp, dh, dw


def check(h, w, t, weight, got, dt, divisor=3.0, temperature=1.0, grad_scale=1.0):
    stats, logp, dh, dw = got
    hd, wd, t = h.double().cpu(), w.double().cpu(), t.cpu()
    n, d = hd.shape
    v = wd.shape[0]
    ok = (t >= 0) & (t < v)
    at = torch.where(ok, t, torch.zeros_like(t))
    x = hd @ wd.T / temperature
    e = (2 * (d / 32 + 8) * U * (hd.abs() @ wd.abs().T) / temperature).max(1).values
    lp = torch.log_softmax(x, 1)
    top = x.max(1, keepdim=True).values
    z = torch.where(top - x < 42, top - x, torch.zeros_like(x)).max(1).values
    said = lp[torch.arange(n), at]
    z = torch.maximum(z, -said)
    r = 2 * e + (6 * z + 40) * U
    want = torch.where(ok, said, torch.zeros_like(said))
    tol = torch.where(ok, r + U * said.abs(), torch.zeros_like(said))
    assert ((logp.double().cpu() - want).abs() <= tol).all(), float(((logp.double().cpu() - want).abs() - tol).max())
    share = (torch.ones(n, dtype=torch.float64) if weight is None else weight.double().cpu()) / divisor * ok
    loss, size = -(share * want).sum(), (share.abs() * tol).sum()
    assert abs(float(stats[0]) - float(loss)) <= float(size) + 2 * U * abs(float(loss))
    assert int(stats[1]) == int(ok.sum())
    coef = share * grad_scale / temperature
    p = lp.exp()
    hot = torch.zeros_like(p)
    hot[torch.arange(n), at] = 1
    # the target's own entry without cancellation, as it is formed
    dx = coef[:, None] * (p - hot)
    dx[torch.arange(n), at] = coef * torch.expm1(said)
    eps = torch.finfo(DT[dt]).eps
    off = (r[:, None] + 1.01 * 2.0 ** -11 + eps / 2) * dx.abs() + 2.0 ** -38 * coef.abs().max()
    off[torch.arange(n), at] = (r + eps / 256) * dx[torch.arange(n), at].abs() + 2.0 ** -38 * coef.abs().max()
    off = off * ok[:, None]
    for name, g, a, k in (("dhidden", dh, wd, v), ("dweight", dw, hd, n)):
        if g is None:
            continue
        m, o = (dx, off) if name == "dhidden" else (dx.T, off.T)
        want = m @ a
        tol = o @ a.abs() + 2 * (k / 32 + 70) * U * (m.abs() @ a.abs())
        tol = tol + (eps / 2) * (want.abs() + tol) + SUB[dt]
        off_by = (g.double().cpu() - want).abs() - tol
        assert not torch.isnan(off_by).any() and float(off_by.max()) <= 0, (name, float(off_by.max()))
    if dh is not None:
        assert (dh.cpu()[~ok] == 0).all()


@pytest.mark.parametrize("temperature", [1.0, 0.7])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("n, v, d, piece", SHAPES)
def test_loss_and_gradients(n, v, d, piece, dt, temperature):
    h, w, t, weight = problem(n, v, d, dt)
    scale = 1024.0 if dt == "f16" else 1.0
    got = run(h, w, t, weight, temperature=temperature, grad_scale=scale, piece=piece)
    check(h, w, t, weight, got, dt, temperature=temperature, grad_scale=scale)
    # without gradients, or with one of them: the same bits
    for grads in ((False, False), (True, False), (False, True)):
        part = run(h, w, t, weight, temperature=temperature, grad_scale=scale, piece=piece, grads=grads)
        for a, b in zip(part, got):
            assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("n, v, d", [(9, 100, 48), (300, 515, 264)])
def test_strides_no_weights_and_nothing_else_written(n, v, d, dt):
    h, w, t, _ = problem(n, v, d, dt, pad=24)
    got = run(h, w, t, None, divisor=float(n), pad=16)
    check(h, w, t, None, got, dt, divisor=float(n))
    for g, m in ((got[2], n), (got[3], v)):
        whole = g.as_strided((m, d + 16), (d + 16, 1))
        assert (whole[:, d:] == 5).all()  # between the rows
    dense = run(h.contiguous(), w.contiguous(), t, None, divisor=float(n))
    for a, b in zip(dense, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("n", [3, 40, 300])
def test_confident_and_hopeless_rows(n, dt):
    """Targets far above and far below everything else: 1 - p without cancellation, rows whose
    target has no probability that fp32 holds."""
    v, d = 700, 64
    h, w, t, weight = problem(n, v, d, dt, spread=1.0, ignore=0.0)
    g = torch.Generator().manual_seed(4)
    sure = torch.arange(n) % 3 == 0
    at = torch.where((t.cpu() >= 0) & (t.cpu() < v), t.cpu(), torch.zeros(n, dtype=torch.int64))
    pull = w.cpu().float()[at] / w.cpu().float()[at].pow(2).sum(1, keepdim=True)
    lift = torch.where(sure, 25.0, -150.0)[:, None] * (1 + 0.1 * torch.rand(n, 1, generator=g))
    h.copy_(h.cpu().float() * 0.3 + pull * lift)
    got = run(h, w, t, weight, grad_scale=64.0)
    check(h, w, t, weight, got, dt, grad_scale=64.0)
    assert float(got[1].min()) < -100


@pytest.mark.parametrize("n", [1, 20, 300])
def test_rows_that_do_not_count(n):
    h, w, t, weight = problem(n, 333, 64, "bf16")
    t.fill_(-100)
    h.fill_(float("nan"))  # unread
    stats, logp, dh, dw = run(h, w, t, weight)
    assert (stats == 0).all() and (logp == 0).all() and (dh == 0).all() and (dw == 0).all()
    # weights of zero: log-probabilities, but no loss and no gradient
    h, w, t, weight = problem(n, 333, 64, "bf16")
    stats, logp, dh, dw = run(h, w, t, torch.zeros_like(weight))
    assert stats[0] == 0 and (logp[(t >= 0) & (t < 333)] < 0).all() and (dh == 0).all() and (dw == 0).all()


def test_no_rows():
    w = torch.randn(50, 16, device=DEV).bfloat16()
    none, t = torch.empty(0, 16, dtype=torch.bfloat16, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV)
    stats, logp, dh, dw = run(none, w, t, None)
    assert (stats == 0).all() and (dw == 0).all()


@pytest.mark.parametrize("n", [5, 200])
def test_weights_of_any_size_and_sign(n):
    h, w, t, weight = problem(n, 600, 72, "bf16")
    weight *= torch.where(torch.arange(n, device=DEV) % 2 == 0, -1.0, 1e-3)
    got = run(h, w, t, weight)
    check(h, w, t, weight, got, "bf16")


@pytest.mark.parametrize("n", [6, 70, 1100])
def test_non_finite_rows_stay_where_they_are(n):
    v, d = 300, 64
    h, w, t, weight = problem(n, v, d, "bf16", ignore=0.0)
    clean = run(h, w, t, weight)
    h[3, 5], h[4, 1] = float("nan"), float("inf")
    bad = run(h, w, t, weight)
    assert torch.isnan(bad[0][0]) and torch.isnan(bad[1][3:5]).all() and torch.isnan(bad[2][3:5]).all()
    rest = [i for i in range(n) if i not in (3, 4)]
    assert torch.equal(bad[1][rest], clean[1][rest]) and torch.equal(bad[2][rest], clean[2][rest])
    assert torch.isnan(bad[3]).all()


def test_same_bits_every_time_and_on_another_stream():
    h, w, t, weight = problem(700, 3000, 264, "bf16")
    ws = zs.linear_cross_entropy_workspace(1000, 3000, 264)  # made for more rows
    first = run(h, w, t, weight, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for k in range(3):
        with torch.cuda.stream(side):
            again = run(h, w, t, weight, ws=ws)
        side.synchronize()
        for a, b in zip(again, first):
            assert torch.equal(a, b), k
        few = run(h[:5], w, t[:5], weight[:5], ws=ws)  # another shape in the same workspace between them
        check(h[:5], w, t[:5], weight[:5], few, "bf16")


@pytest.mark.parametrize("n", [8, 300])
def test_captured_and_replayed(n):
    """A graph of the forward and backward calls, replayed with eager calls between."""
    v, d = 1000, 128
    h, w, t, weight = problem(n, v, d, "bf16")
    ws, ews = (zs.linear_cross_entropy_workspace(n, v, d) for _ in range(2))
    nws, gws = zs.rms_norm_workspace(n, d), zs.embedding_workspace(n, v, d)
    gain = torch.ones(d, dtype=torch.bfloat16, device=DEV)
    f = lambda *s: torch.zeros(*s, device=DEV)  # noqa: E731
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    tokens = torch.arange(n, device=DEV) * 7 % v

    def step(head_ws, o):
        zs.zero_embedding(w, tokens, o["x"], scale=2.0)
        zs.zero_rms_norm(o["x"], gain, o["y"], residual=h, h=o["h"], rstd=o["rstd"], codes=o["codes"], scales=o["scales"])
        zs.zero_linear_cross_entropy(o["y"], w, t, row_weight=weight, divisor=3.0, stats=o["stats"], logp=o["logp"],
                                     dhidden=o["dy"], dweight=o["dw"], workspace=head_ws)
        zs.zero_rms_norm_backward(o["dy"], gain, o["rstd"], o["dx"], o["dgain"], codes=o["codes"], scales=o["scales"],
                                  workspace=nws)
        zs.zero_embedding_grad(o["dx"], tokens, o["dw"], scale=2.0, accumulate=True, workspace=gws)

    def outputs():
        return dict(x=b(n, d), y=b(n, d), h=b(n, d), rstd=f(n), codes=torch.zeros(n, d, dtype=torch.float8_e4m3fn, device=DEV),
                    scales=f(n, 1), stats=f(2), logp=f(n), dy=b(n, d), dw=b(v, d), dx=b(n, d), dgain=b(d))

    eager, o = outputs(), outputs()
    step(ews, eager)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(ws, o)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(ws, o)
    for _ in range(4):
        for x in o.values():
            x.zero_()
        graph.replay()
        step(ews, eager)
        torch.cuda.synchronize()
        for k in o:
            assert torch.equal(o[k].float(), eager[k].float()), k
        h.mul_(1.01)  # other inputs for the next replay


def test_gradients_against_differences():
    """Along random directions, against the change of the loss in 64 bits; the gradients' own
    rounding (11 bits and bf16's half step on either side) allowed for by magnitudes."""
    n, v, d = 40, 90, 64
    h, w, t, weight = problem(n, v, d, "bf16")
    _, _, dh, dw = run(h, w, t, weight)
    hd, wd, t, weight = h.double().cpu(), w.double().cpu(), t.cpu(), weight.double().cpu()
    ok = (t >= 0) & (t < v)

    def loss(a, b):
        lp = torch.log_softmax(a @ b.T, 1)
        return -(weight[ok] * lp[ok, t[ok]]).sum() / 3.0

    p = (hd @ wd.T).softmax(1)
    hot = torch.zeros_like(p)
    hot[ok, t[ok]] = 1
    mags = (weight * ok / 3.0)[:, None] * (p - hot).abs()
    room = (2.0 ** -11 + 2.0 ** -8 + 2.0 ** -8) * 1.1  # of dx's two roundings and the gradient's own
    gen = torch.Generator().manual_seed(2)
    for _ in range(5):
        a = torch.randn(n, d, generator=gen, dtype=torch.float64)
        b = torch.randn(v, d, generator=gen, dtype=torch.float64)
        s = 1e-5
        slope = (loss(hd + s * a, wd + s * b) - loss(hd - s * a, wd - s * b)) / (2 * s)
        got = (dh.double().cpu() * a).sum() + (dw.double().cpu() * b).sum()
        size = ((mags @ wd.abs()) * a.abs()).sum() + ((mags.T @ hd.abs()) * b.abs()).sum()
        assert abs(got - slope) <= 2 * room * size + 1e-7 * size


def test_binding_refuses():
    h, w, t, weight = problem(5, 40, 16, "bf16")
    ws = zs.linear_cross_entropy_workspace(5, 40, 16)
    good = dict(hidden=h, weight=w, targets=t, divisor=1.0, stats=torch.zeros(2, device=DEV), logp=torch.zeros(5, device=DEV),
                workspace=ws)
    for bad in (dict(hidden=h.float()), dict(weight=w.half()), dict(hidden=h[:, :8]), dict(targets=t[:3]), dict(targets=t.int()),
                dict(logp=torch.zeros(4, device=DEV)), dict(dhidden=h[:3]), dict(dweight=w.float()), dict(hidden=h.t()),
                dict(row_weight=weight[:2]), dict(stats=torch.zeros(1, device=DEV)), dict(hidden=h[0])):
        with pytest.raises((ValueError, TypeError)):
            zs.zero_linear_cross_entropy(**{**good, **bad})
    for bad in (dict(hidden=h.float(), weight=w.float()), dict(workspace=ws[:512]), dict(divisor=0.0), dict(piece_rows=0),
                dict(dhidden=torch.zeros(5, 20, dtype=h.dtype, device=DEV)[:, 1:17]),
                dict(hidden=h[:, :12].contiguous(), weight=w[:, :12].contiguous())):
        with pytest.raises(zs.ZeroShardError):
            zs.zero_linear_cross_entropy(**{**good, **bad})
