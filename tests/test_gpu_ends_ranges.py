"""The embedding, norm and linear cross entropy calls over ranges that their own files leave
out: workspaces made for other sizes, long sums, weights of very different sizes."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import zero_sharded_optimizer_owned_amd as zs  # noqa: E402
import test_gpu_embedding as emb  # noqa: E402
import test_gpu_head as head  # noqa: E402

DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    zs.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("accumulate", [False, True])
def test_short_batches_in_the_workspace_of_a_long_one(accumulate):
    """One workspace made for 5000 tokens, with its contents left by the batch before."""
    v, d = 700, 72
    ws = zs.embedding_workspace(5000, v, d)
    for n in (5000, 4096, 300, 4097, 1041, 1, 4095, 1024):
        dout = torch.randn(n, d, generator=torch.Generator().manual_seed(n)).bfloat16().to(DEV)
        tokens = emb.tokens_of(n, v, 3)
        dtable, _ = emb.table_of(v, d, 0, "bf16", 9)
        start = dtable.clone()
        zs.zero_embedding_grad(dout, tokens, dtable, workspace=ws, scale=0.3, accumulate=accumulate)
        want, tol, _ = emb.grad_reference(dout, tokens, v, 0.3, start if accumulate else None)
        emb.within(dtable, want, tol + emb.half_step(want, "bf16"))


@pytest.mark.parametrize("dt, out", [("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("n", [4000, 20_000, 200_000, 400_001])
def test_long_runs_of_one_token(n, dt, out):
    """Three quarters of the positions name one token (unmasked padding).  A sum of c rows is
    chains of at most 32 additions in fp32, added in fp64 and rounded once: (min(c, 32) + 1) u
    of the magnitudes, and the scale with its product 2 u of the result."""
    d, v = 9, 60
    g = torch.Generator().manual_seed(n)
    tokens = torch.randint(0, v, (n,), generator=g)
    tokens[torch.rand(n, generator=g) < 0.75] = 7
    dout = (1 + torch.rand(n, d, generator=g)).to(emb.DT[dt])
    if dt == "f32":
        dout[:, 0] = 1 + 2.0 ** -13  # 32 of them add up to 32 + 2^-8, which a sum past 2^17 cannot take
    dtable = torch.empty(v, d, dtype=emb.DT[out], device=DEV)
    zs.zero_embedding_grad(dout.to(DEV), tokens.to(DEV), dtable, workspace=zs.embedding_workspace(n, v, d), scale=0.3)
    want, _, _ = emb.grad_reference(dout, tokens, v, 0.3, None)
    count = torch.bincount(tokens, minlength=v).double()[:, None]
    emb.within(dtable, want, ((count.clamp(max=32) + 1) + 2) * U * want + emb.half_step(want, out))


@pytest.mark.parametrize("grads", ["both", "dhidden"])
@pytest.mark.parametrize("n, v, d", [(5, 46_811, 64), (40, 46_811, 64), (300, 46_811, 16), (1100, 30_011, 8), (290, 1999, 600)])
def test_a_row_s_gradient_does_not_depend_on_other_rows_weights(n, v, d, grads):
    """fp16, row weights from 1 down to 2^-22 of it, dhidden in one part of the vocabulary and in
    several.  A row keeps softmax - onehot in steps of at most 2^-30 (2^-24 / (2^14 2^-8)), so to
    half of that, and its exponentials down to 2^-40: 2^-30 of the row's own factor holds both,
    where what test_gpu_head.py allows is 2^-38 of the largest one."""
    h, w, t, _ = head.problem(n, v, d, "f16", spread=0.3 * d ** 0.5)
    w += 0.5  # a mean: what is lost of many small probabilities does not average out
    size = torch.tensor([1.0, 2.0 ** -22, -2.0 ** -7, 2.0 ** -9, -2.0 ** -15, 0.0, 1.3 * 2.0 ** -20, 2.0 ** -21])
    i = torch.arange(n)
    weight = size[torch.where(i < 2, i, (i * 5 + 1) % 8)].to(DEV)
    h[weight.abs() < 2.0 ** -8] = 0  # equal probabilities
    t[1] = v // 3
    args = dict(divisor=1.0, grad_scale=2.0 ** 10)
    got = head.run(h, w, t, weight, grads=(True, grads == "both"), **args)
    head.check(h, w, t, weight, got, "f16", **args)
    if grads == "both":  # dweight alone: the same bits
        alone = head.run(h, w, t, weight, grads=(False, True), **args)
        assert torch.equal(alone[3], got[3])
    hd, wd, at, coef = h.double().cpu(), w.double().cpu(), t.cpu(), weight.double().cpu() * 2.0 ** 10
    ok = (at >= 0) & (at < v)
    hd, at, coef, row = hd[ok], at[ok], coef[ok], torch.arange(int(ok.sum()))
    x = hd @ wd.T
    lp = torch.log_softmax(x, 1)
    e = (2 * (d / 32 + 8) * U * (hd.abs() @ wd.abs().T)).max(1).values
    r = 2 * e + (6 * (x.max(1).values - x.min(1).values) + 40) * U
    dx = lp.exp()
    dx[row, at] = torch.expm1(lp[row, at])
    off = (r[:, None] + 2.01 * 2.0 ** -11) * dx.abs() + 2.0 ** -30
    off[row, at] = (r + 2.0 ** -18) * dx[row, at].abs() + 2.0 ** -30
    want = coef[:, None] * (dx @ wd)
    tol = coef.abs()[:, None] * (off @ wd.abs() + 2 * (v / 32 + 70) * U * (dx.abs() @ wd.abs()))
    emb.within(got[2][ok.to(DEV)], want, tol + 2.0 ** -11 * (want.abs() + tol) + 2.0 ** -25)


@pytest.mark.parametrize("n", [30_720, 32_768, 32_769, 34_817])
def test_gradient_at_the_number_of_blocks_that_a_sort_scans(n):
    v, d = 5000, 8
    dout = torch.randn(n, d, generator=torch.Generator().manual_seed(n)).to(DEV)
    tokens = emb.tokens_of(n, v, 3)
    dtable = torch.empty(v, d, device=DEV)
    zs.zero_embedding_grad(dout, tokens, dtable, workspace=zs.embedding_workspace(n, v, d))
    want, tol, _ = emb.grad_reference(dout, tokens, v, 1.0, None)
    emb.within(dtable, want, tol + emb.half_step(want, "f32"))


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n, v, d", [(9, 5, 7), (333, 1000, 100), (9000, 70, 33)])
def test_half_precision_into_an_fp32_table(n, v, d, accumulate):
    dout = torch.randn(n, d, generator=torch.Generator().manual_seed(n)).half().to(DEV)
    tokens = emb.tokens_of(n, v, 3)
    dtable, _ = emb.table_of(v, d, d + 3, "f32", 9)
    start = dtable.clone()
    zs.zero_embedding_grad(dout, tokens, dtable, workspace=zs.embedding_workspace(n, v, d), scale=0.3, accumulate=accumulate)
    want, tol, _ = emb.grad_reference(dout, tokens, v, 0.3, start if accumulate else None)
    emb.within(dtable, want, tol + emb.half_step(want, "f32"))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("piece", [8192, 300, 6])
def test_weights_of_all_sizes_in_pieces(piece, dt):
    """Pieces whose largest weights differ, one of them with small weights alone."""
    n, v, d = 700, 5001, 40
    h, w, t, _ = head.problem(n, v, d, dt)
    i = torch.arange(n)
    weight = (torch.where(i % 3 == 0, 2.0 ** -13, 1.0) * torch.where(i >= 300, 1.0, 2.0 ** -20)).to(DEV)
    got = head.run(h, w, t, weight, piece=piece, grad_scale=2.0 ** 9)
    head.check(h, w, t, weight, got, dt, grad_scale=2.0 ** 9)
    # a negligible row's weight: the same log-probabilities, and the others' gradients to the bit
    weight[1] = 0.0
    again = head.run(h, w, t, weight, piece=piece, grad_scale=2.0 ** 9)
    assert torch.equal(again[1], got[1]) and torch.equal(again[2][2:], got[2][2:])


def test_weights_that_are_not_finite_beside_small_ones():
    """fp16: a row of infinite weight is NaN or infinite by itself, the others' gradients are not."""
    n, v, d = 40, 700, 64
    h, w, t, weight = head.problem(n, v, d, "f16", ignore=0.0)
    weight[::2] *= 2.0 ** -14
    clean = head.run(h, w, t, weight, grad_scale=2.0 ** 9)
    top = int(weight.argmax())
    k = 5 if top != 5 else 7
    weight[k] = float("inf")
    got = head.run(h, w, t, weight, grad_scale=2.0 ** 9)
    rest = [i for i in range(n) if i != k]
    assert torch.equal(got[2][rest], clean[2][rest]) and torch.equal(got[1], clean[1])
    assert not torch.isfinite(got[2][k]).any() and not torch.isfinite(got[0][0])


@pytest.mark.parametrize("piece", [8192, 70])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("n, v, d", [(1, 3, 8), (2, 2017, 8), (3, 220, 16), (8, 500, 264), (9, 500, 24), (45, 371, 384),
                                     (64, 1500, 136), (64, 5001, 520), (65, 300, 16), (128, 900, 16), (129, 257, 8),
                                     (190, 1550, 8), (300, 5001, 16), (1030, 700, 16), (1100, 3278, 8)])
def test_small_heads_in_two_numbers(n, v, d, dt, weighted, piece):
    """Up to 64 rows and up to dim 16 softmax - onehot is held in two numbers of the type.  The exponentials' two of
    11 bits are off by 2^-24, dx's by 2^-24 (fp16) or 2^-18 (bf16: half a step of 8 bits, twice),
    all relative; what is below fp16's smallest numbers by 2^-38 of the largest factor."""
    if piece == 70 and n < 128:
        return
    h, w, t, weight = head.problem(n, v, d, dt, spread=4.0)
    if weighted:
        weight *= torch.where(torch.arange(n, device=DEV) % 2 == 0, -1.0, 2.0 ** -9)
    else:
        weight = None
    scale = 2.0 ** 7 if dt == "f16" else 1.0
    got = head.run(h, w, t, weight, temperature=0.8, grad_scale=scale, piece=piece)
    head.check(h, w, t, weight, got, dt, temperature=0.8, grad_scale=scale)
    for grads in ((True, False), (False, True)):
        part = head.run(h, w, t, weight, temperature=0.8, grad_scale=scale, piece=piece, grads=grads)
        for a, b in zip(part, got):
            assert a is None or torch.equal(a, b)
    hd, wd, at = h.double().cpu(), w.double().cpu(), t.cpu()
    ok = (at >= 0) & (at < v)
    hd, at, row = hd[ok], at[ok], torch.arange(int(ok.sum()))
    coef = (torch.ones(n, dtype=torch.float64) if weight is None else weight.double().cpu())[ok] * scale / 3.0 / 0.8
    x = hd @ wd.T / 0.8
    lp = torch.log_softmax(x, 1)
    e = (2 * (d / 32 + 8) * U * (hd.abs() @ wd.abs().T) / 0.8).max(1).values
    z = torch.maximum((x.max(1).values - x.min(1).values).clamp(max=42), -lp[row, at])
    r = 2 * e + (6 * z + 40) * U
    dx = coef[:, None] * lp.exp()
    dx[row, at] = coef * torch.expm1(lp[row, at])
    eps = torch.finfo(emb.DT[dt]).eps
    off = (r[:, None] + 2 * U + (2.0 ** -18 if dt == "bf16" else U)) * dx.abs() + 2.0 ** -38 * coef.abs().max()
    for g, m, o, a, k in ((got[2][ok.to(DEV)], dx, off, wd, v), (got[3], dx.T, off.T, hd, n)):
        want = m @ a
        tol = o @ a.abs() + 2 * (2 * k / 32 + 70) * U * (m.abs() @ a.abs())
        emb.within(g, want, tol + (eps / 2) * (want.abs() + tol) + head.SUB[dt])


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("d", [1, 2, 3, 9])
def test_norm_of_few_columns_cancels_what_cancels(d, keep):
    """With one column n = h rstd is near 1 and dx = rstd dy gain (1 - n^2) far less than its two
    terms, so that e = dy gain has to be the same number in both: as fp32 has n and e, dx is off by
    the roundings of up to 8 sums of e n (fused: u each of their magnitudes), of the mean (u; of
    one column none) and by 3 u of itself (the difference is fused)."""
    n = 4000
    g = torch.Generator().manual_seed(d)
    x, dy, gain = (torch.randn(*s, generator=g).to(DEV) for s in ((n, d), (n, d), (d,)))
    rstd = torch.empty(n, device=DEV)
    codes, scales = torch.empty(n, d, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(n, 1, device=DEV)
    zs.zero_rms_norm(x, gain, torch.empty_like(x), rstd=rstd, codes=codes, scales=scales)
    held = dict(codes=codes, scales=scales) if keep else dict(h=x)
    dx, dgain = torch.empty_like(x), torch.empty_like(gain)
    zs.zero_rms_norm_backward(dy, gain, rstd, dx, dgain, workspace=zs.rms_norm_workspace(n, d), **held)
    # from what the kernel reads, with n and dy gain as fp32 has them, the rest in 64 bits
    h = codes.float() * scales if keep else x
    norm, e = (h * rstd[:, None]).double(), (dy * gain).double()
    r = rstd.double()[:, None]
    m = (e * norm).mean(1, keepdim=True)
    want = r * (e - norm * m)
    tol = U * r * norm.abs() * ((e * norm).abs().mean(1, keepdim=True) * min(d, 8) + (m.abs() if d > 1 else 0)) + 3 * U * want.abs()
    emb.within(dx, want.cpu(), tol.cpu() + 2.0 ** -150)


@pytest.mark.parametrize("n, d", [(40, 136), (300, 136), (300, 8)])
def test_rows_of_small_weight_captured_and_on_two_streams(n, d):
    """fp16 with lifted rows, in one number and in two: a graph replayed with eager calls between
    and other inputs, and two calls at once in a workspace each, to the bit."""
    v = 5001
    h, w, t, weight = head.problem(n, v, d, "f16")
    weight *= torch.where(torch.arange(n, device=DEV) % 2 == 0, 1.0, 2.0 ** -14)

    def buffers():
        return (torch.zeros(2, device=DEV), torch.zeros(n, device=DEV), torch.zeros_like(h), torch.zeros_like(w),
                zs.linear_cross_entropy_workspace(n, v, d))

    def call(b, x):
        zs.zero_linear_cross_entropy(x, w, t, row_weight=weight, divisor=2.0, grad_scale=2.0 ** 9, stats=b[0], logp=b[1],
                                     dhidden=b[2], dweight=b[3], workspace=b[4])

    eager, held, other = buffers(), buffers(), buffers()
    call(held, h)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(held, h)
    for _ in range(3):
        for x in held[:4]:
            x.zero_()
        graph.replay()
        call(eager, h)
        torch.cuda.synchronize()
        for a, b in zip(held[:4], eager[:4]):
            assert torch.equal(a, b)
        h.mul_(0.9)
    h2 = h * 0.5
    call(eager, h2)
    want = [x.clone() for x in eager[:4]]
    call(eager, h)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s, b, x in zip(streams, (held, other), (h, h2)):
            with torch.cuda.stream(s):
                call(b, x)
    torch.cuda.synchronize()
    for a, b in zip(held[:4], eager[:4]):
        assert torch.equal(a, b)
    for a, b in zip(other[:4], want):
        assert torch.equal(a, b)
