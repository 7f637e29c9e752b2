"""The embedding lookup and its gradient against their definitions in 64 bits.

Tolerances.  u = 2^-24.  A looked-up value carries the rounding of the scale
and of the product, 2 u relative, and the store's half step.  A gradient's
sum of c rows is a chain of at most 32 additions and one of at most
c / 8 + 1 partial sums, so it is off by at most (min(c, 32) + c / 8 + 1) u
times the sum of magnitudes; the scale, its product and the addition to the old
gradient add 3 u, the store half a step (or half the smallest subnormal).
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import zero_sharded_optimizer_owned_amd as zs  # noqa: E402

DEV = "cuda"
U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SUB = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}
#         tokens, vocab, dim, table row stride (0: dense)
SHAPES = [(1, 1, 1, 0), (1, 7, 8, 0), (2, 3, 9, 11), (5, 10, 3, 0), (64, 4, 16, 0), (65, 300, 31, 40), (333, 1000, 100, 0),
          (1000, 17, 257, 0), (4095, 513, 64, 0), (4097, 50_001, 33, 0), (16_384, 262_143, 5, 0), (16_385, 900, 24, 25),
          (20_000, 3, 40, 0), (33_000, 600_000, 4, 0), (700, 90, 5003, 0), (40, 12, 20_000, 0),
          (1024, 90, 12, 0), (1025, 90, 12, 0), (8192, 300, 20, 0), (8193, 300, 20, 0), (131_072, 70_000, 3, 0), (131_073, 40, 4, 0),
          (700_001, 1000, 2, 0)]


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


def table_of(v, d, stride, dt, seed=0, fill=None):
    """[v, d] at a row stride inside a larger buffer, and that buffer."""
    g = torch.Generator().manual_seed(seed + v + 7 * d)
    stride = stride or d
    buf = torch.full((v * stride + 16,), 5.0, dtype=DT[dt], device=DEV)
    t = buf[1:1 + v * stride].view(v, stride)[:, :d]  # at an odd element
    t.copy_(torch.randn(v, d, generator=g) if fill is None else torch.full((v, d), fill))
    return t, buf


def tokens_of(n, v, seed=0, skew=True):
    """Some outside the table, some tokens far more frequent than others."""
    g = torch.Generator().manual_seed(seed + n)
    t = torch.randint(0, v, (n,), generator=g)
    if skew and n > 3:
        t[torch.rand(n, generator=g) < 0.4] = v // 2
        t[torch.rand(n, generator=g) < 0.1] = -1
        t[n // 2] = v
        t[n // 3] = 2 ** 40
    return t.to(DEV)


def grad_reference(dout, tokens, v, scale, start):
    dout, t = dout.double().cpu(), tokens.cpu()
    ok = (t >= 0) & (t < v)
    t, d = t[ok], dout[ok]
    total = torch.zeros(v, dout.shape[1], dtype=torch.float64).index_add_(0, t, d)
    mags = torch.zeros_like(total).index_add_(0, t, d.abs())
    count = torch.bincount(t, minlength=v).double()[:, None]
    want = total * scale + (0 if start is None else start.double().cpu())
    chain = count.clamp(max=32) + count / 8 + 1
    tol = (chain + 3) * U * mags * abs(scale) + 2 * U * want.abs()
    return want, tol, count[:, 0] > 0


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("n, v, d, stride", SHAPES)
def test_lookup(n, v, d, stride, dt):
    table, _ = table_of(v, d, stride, dt)
    tokens = tokens_of(n, v)
    out = torch.full((n, d), 9.0, dtype=DT[dt], device=DEV)
    zs.zero_embedding(table, tokens, out, scale=1.7)
    t = tokens.cpu()
    ok = (t >= 0) & (t < v)
    want = torch.where(ok[:, None], table.double().cpu()[torch.where(ok, t, torch.zeros_like(t))] * 1.7, 0.0)
    within(out, want, 2 * U * want.abs() + half_step(want, dt))
    assert (out.cpu()[~ok] == 0).all()
    one = torch.empty_like(out)
    zs.zero_embedding(table, tokens, one)
    assert torch.equal(one[ok.to(DEV)], table[tokens[ok.to(DEV)]])


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dt, out", [("f16", "f16"), ("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("n, v, d, stride", SHAPES)
def test_gradient(n, v, d, stride, dt, out, accumulate):
    g = torch.Generator().manual_seed(n * 31 + d)
    dout = torch.randn(n, d, generator=g).to(DT[dt]).to(DEV)
    tokens = tokens_of(n, v, 5)
    dtable, buf = table_of(v, d, stride, out, 9, None if accumulate else float("nan"))
    start, around = dtable.clone(), buf.clone()
    ws = zs.embedding_workspace(n, v, d)
    ws.fill_(0xA5)  # its contents do not matter
    zs.zero_embedding_grad(dout, tokens, dtable, workspace=ws, scale=0.3, accumulate=accumulate)
    want, tol, named = grad_reference(dout, tokens, v, 0.3, start if accumulate else None)
    within(dtable, want, tol + half_step(want, out))
    if accumulate:
        assert torch.equal(dtable[~named.to(DEV)], start[~named.to(DEV)])
    else:
        assert (dtable[~named.to(DEV)] == 0).all()
    # nothing outside the rows
    dtable.copy_(start)
    assert torch.equal(torch.nan_to_num(buf, 3.0), torch.nan_to_num(around, 3.0))


@pytest.mark.parametrize("n", [1, 8, 9, 300, 5000, 20_000])
def test_gradient_of_one_token_only(n):
    """Every position names the same token: one run over all tiles."""
    dout = torch.randn(n, 72, generator=torch.Generator().manual_seed(n)).to(DEV)
    tokens = torch.full((n,), 3, dtype=torch.int64, device=DEV)
    dtable = torch.empty(5, 72, device=DEV)
    zs.zero_embedding_grad(dout, tokens, dtable, workspace=zs.embedding_workspace(n, 5, 72))
    want, tol, _ = grad_reference(dout, tokens, 5, 1.0, None)
    within(dtable, want, tol + half_step(want, "f32"))


@pytest.mark.parametrize("n", [0, 7])
def test_gradient_of_no_token(n):
    dtable = torch.full((6, 10), 2.0, device=DEV)
    dout, tokens = torch.randn(n, 10, device=DEV), torch.full((n,), -1, dtype=torch.int64, device=DEV)
    ws = zs.embedding_workspace(n, 6, 10)
    zs.zero_embedding_grad(dout, tokens, dtable, workspace=ws, accumulate=True)
    assert (dtable == 2).all()
    zs.zero_embedding_grad(dout, tokens, dtable, workspace=ws)
    assert (dtable == 0).all()
    out = torch.full((n, 10), 3.0, device=DEV)
    zs.zero_embedding(dtable, tokens, out)
    assert (out == 0).all()


@pytest.mark.parametrize("n", [3000, 17_000])
def test_gradient_is_the_same_every_time_and_in_pieces_of_the_order(n):
    """Bit for bit the same from run to run; an fp32 sum in which order matters."""
    g = torch.Generator().manual_seed(1)
    dout = (torch.randn(n, 40, generator=g) * torch.logspace(-6, 6, n)[:, None]).to(DEV)
    tokens = tokens_of(n, 50)
    ws = zs.embedding_workspace(n, 50, 40)
    first = None
    for _ in range(4):
        dtable = torch.empty(50, 40, device=DEV)
        zs.zero_embedding_grad(dout, tokens, dtable, workspace=ws)
        assert first is None or torch.equal(first, dtable)
        first = dtable


def test_gradient_of_infinities_stays_in_its_rows():
    dout = torch.ones(40, 8, device=DEV)
    dout[3], dout[7] = float("inf"), float("nan")
    tokens = torch.arange(40, device=DEV) % 10
    dtable = torch.empty(10, 8, device=DEV)
    zs.zero_embedding_grad(dout, tokens, dtable, workspace=zs.embedding_workspace(40, 10, 8))
    assert torch.isinf(dtable[3]).all() and torch.isnan(dtable[7]).all()
    rest = [i for i in range(10) if i not in (3, 7)]
    assert (dtable[rest] == 4).all()


def test_table_past_32_bit_offsets():
    """Rows whose byte offset is beyond 2^32."""
    v, d = 1_100_000, 2048
    table = torch.zeros(v, d, dtype=torch.bfloat16, device=DEV)
    tokens = torch.tensor([v - 1, 0, 1_050_000, v - 1], device=DEV)
    table[v - 1], table[1_050_000] = 2.0, 3.0
    out = torch.empty(4, d, dtype=torch.bfloat16, device=DEV)
    zs.zero_embedding(table, tokens, out)
    assert out[:, 0].tolist() == [2.0, 0.0, 3.0, 2.0] and torch.equal(out, table[tokens])
    table.fill_(float("nan"))
    zs.zero_embedding_grad(out, tokens, table, workspace=zs.embedding_workspace(4, v, d))
    assert table[v - 1, 5] == 4 and table[1_050_000, d - 1] == 3 and table[0, 0] == 0
    table[v - 1] = table[1_050_000] = 0
    assert not table.any()


def test_binding_refuses():
    table, out = torch.zeros(5, 8, device=DEV), torch.zeros(3, 8, device=DEV)
    t, ws = torch.zeros(3, dtype=torch.int64, device=DEV), zs.embedding_workspace(3, 5, 8)
    for bad in (dict(table=table.double()), dict(table=table[:, ::2]), dict(tokens=t.int()), dict(out=out[:2]),
                dict(out=out.half()), dict(table=table[0]), dict(out=out.t())):
        with pytest.raises((ValueError, TypeError, KeyError)):
            zs.zero_embedding(**{**dict(table=table, tokens=t, out=out), **bad})
    for bad in (dict(dout=out[:2]), dict(dtable=table.t()), dict(dtable=table[:, :7]), dict(tokens=t.cpu()),
                dict(workspace=ws.cpu())):
        with pytest.raises((ValueError, TypeError)):
            zs.zero_embedding_grad(**{**dict(dout=out, tokens=t, dtable=table, workspace=ws), **bad})
    with pytest.raises(zs.ZeroShardError):
        zs.zero_embedding_grad(out, t, table, workspace=ws[:256])
    with pytest.raises(zs.ZeroShardError):
        zs.zero_embedding_grad(out, t, table.half(), workspace=ws)
