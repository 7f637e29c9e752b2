"""The embedding, norm and linear cross entropy calls over ranges that their own files leave
out: workspaces made for other sizes, long sums, weights of very different sizes."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import zero_sharded_optimizer_owned_amd as zs  # noqa: E402
import test_gpu_embedding as emb  # noqa: E402

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
