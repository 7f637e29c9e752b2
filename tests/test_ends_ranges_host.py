"""Workspaces of the embedding, norm and linear cross entropy calls over ranges of sizes, on
the CPU: host calls and argument checks only, nothing is launched."""
import ctypes as ct

import numpy as np
import pytest

import zero_sharded_optimizer_owned_amd as zs

P = 4096  # an address that passes every check (none is looked at on the host)


def size(fn, *args):
    out = np.zeros(1, dtype=np.uint64)
    assert fn(*args, out.ctypes.data) == zs.ZERO_OK
    return int(out[0])


def steps(most, seed):
    """Counts up to `most`: small ones, both sides of powers of two, and some between."""
    near = [(1 << k) + j for k in range(most.bit_length()) for j in (-1, 0, 1)]
    between = np.exp(np.random.RandomState(seed).uniform(0, np.log(most), 200)).astype(int).tolist()
    return sorted({n for n in [*range(70), *near, 1040, 5000, 16_160, *between] if n <= most})


@pytest.mark.parametrize("dim", [1, 8, 9, 1000, 4096, 20_000])
def test_a_workspace_of_the_embedding_gradient_serves_fewer_tokens_and_columns(dim):
    fn = zs.lib().zero_embedding_workspace_bytes
    last = 0
    for n in steps(1 << 28, dim):
        now = size(fn, n, dim)
        assert now >= last and now >= size(fn, n, max(1, dim - 1)) and now >= size(fn, n, max(1, dim // 3)), n
        last = now


def test_the_largest_batch_s_workspace_passes_a_short_one_s_check():
    """The check of the size, seen by the one behind it: workspaces are 256-byte aligned."""
    L = zs.lib()
    a = zs.EmbeddingGradArgs()
    for k, v in dict(dout=P, dtype=zs.ZERO_BF16, tokens=P, vocab=100, dim=4096, scale=1.0, dtable=P,
                     table_dtype=zs.ZERO_BF16, stride=4096, workspace=P + 64,
                     workspace_bytes=size(L.zero_embedding_workspace_bytes, 8192, 4096)).items():
        setattr(a, k, v)
    for n in (1, 333, 4095, 4096, 4097, 8192):
        a.n_tokens = n
        assert L.zero_embedding_grad(ct.byref(a), None) == zs.ZERO_EINVAL
        assert "256-byte" in L.zero_last_error().decode(), n
    a.n_tokens = 8500
    assert L.zero_embedding_grad(ct.byref(a), None) == zs.ZERO_EINVAL and "needs" in L.zero_last_error().decode()


@pytest.mark.parametrize("dim", [1, 9, 5003, 16_384])
def test_a_workspace_of_the_norm_s_backward_pass_serves_fewer_rows_and_columns(dim):
    fn = zs.lib().zero_rms_norm_workspace_bytes
    last = 0
    for n in steps(1 << 30, dim):
        now = size(fn, n, dim)
        assert now >= last and now >= size(fn, n, max(1, dim - 1)) and now >= size(fn, n, max(1, dim // 3)), n
        last = now


@pytest.mark.parametrize("grad", [0, 1])
@pytest.mark.parametrize("vocab, dim, piece", [(200, 8, 8192), (5001, 16, 300), (5001, 24, 300), (60_000, 16, 16_384), (5001, 72, 50), (16_544, 1936, 8192), (32_000, 1088, 300), (128_000, 4096, 16_384),
                                               (50_001, 1000, 5)])
def test_a_workspace_of_the_linear_cross_entropy_serves_fewer_rows(vocab, dim, piece, grad):
    fn = zs.lib().zero_linear_cross_entropy_workspace_bytes
    last = 0
    for n in steps(100_000, vocab):
        now = size(fn, n, vocab, dim, piece, grad)
        assert now >= last and now >= size(fn, n, vocab, dim, piece, 0), n
        last = now


@pytest.mark.parametrize("n", [1, 77, 256, 2202, 8192, 20_000])
@pytest.mark.parametrize("vocab, dim", [(16_544, 1936), (16_544, 2096), (32_000, 64), (32_000, 1024), (32_000, 4096), (50_001, 1000),
                                        (128_000, 4096), (128_000, 16_384), (1 << 20, 8), (1000, 32_768)])
def test_what_a_workspace_of_the_linear_cross_entropy_holds(n, vocab, dim):
    """Two bytes a logit of a piece (four up to 64 rows or dim 16), the hidden states, the tiles' statistics, a few bytes a row, at
    most 512 MiB for the parts of dhidden's sums, and past one piece the sums of dweight."""
    fn = zs.lib().zero_linear_cross_entropy_workspace_bytes
    piece = min(n, 8192)
    padded = -(-vocab // 256) * 256
    # up to 8 rows the statistics are of 16 columns: 8 rows' are 0.5 bytes a logit
    scores = piece * dim * 2 + max(piece * padded // 256, min(piece, 8) * padded // 16) * 8 + 9 * n + 64 * piece + 8192
    assert size(fn, n, vocab, dim, 8192, 0) <= scores
    held = 2 * piece if dim <= 16 else max(piece, 2 * min(piece, 64))
    whole = scores + held * (padded + dim) * 2 + (512 << 20) + (vocab * dim * 4 if n > piece else 0)
    assert held * vocab * 2 <= size(fn, n, vocab, dim, 8192, 1) <= whole
