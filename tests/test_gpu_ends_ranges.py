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
