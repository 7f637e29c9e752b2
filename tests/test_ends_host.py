"""The refusals and workspace sizes of the embedding, norm and linear cross entropy calls,
on the CPU: host calls and argument checks only, nothing is launched."""
import ctypes as ct
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

import zero_sharded_optimizer_owned_amd as zs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 4096  # an address that passes every check (none is looked at on the host)
NAN, INF = float("nan"), float("inf")


def refused(rc, word):
    assert rc == zs.ZERO_EINVAL
    assert word in zs.lib().zero_last_error().decode(), zs.lib().zero_last_error()


def made(kind, good, changes):
    a = kind()
    for k, v in {**good, **changes}.items():
        setattr(a, k, v)
    return ct.byref(a)


def size(fn, *args):
    out = np.zeros(1, dtype=np.uint64)
    assert fn(*args, out.ctypes.data) == zs.ZERO_OK
    return int(out[0])


# table, dtype, vocab, dim, stride, tokens, n_tokens, scale, out
EMBED = [P, zs.ZERO_BF16, 100, 16, 16, P, 5, 1.0, P, None]


@pytest.mark.parametrize("at, bad, word", [
    (0, None, "table"), (0, P + 1, "aligned"), (1, 0, "dtype"), (1, 4, "dtype"), (2, 0, "vocab"), (2, 1 << 31, "vocab"),
    (3, 0, "dim"), (3, (1 << 20) + 1, "dim"), (4, 15, "overlap"), (5, None, "tokens"), (5, P + 4, "aligned"),
    (6, 1 << 62, "overflows"), (7, NAN, "scale"), (7, INF, "scale"), (7, 1e39, "scale"), (8, None, "out"), (8, P + 1, "aligned"),
    (4, 1 << 62, "overflows"),
])
def test_embedding_refuses(at, bad, word):
    refused(zs.lib().zero_embedding(*[bad if i == at else x for i, x in enumerate(EMBED)]), word)


def test_embedding_of_no_tokens_does_nothing():
    assert zs.lib().zero_embedding(P, zs.ZERO_F32, 100, 16, 16, None, 0, 1.0, None, None) == zs.ZERO_OK


EMBED_GRAD = dict(dout=P, dtype=zs.ZERO_F16, tokens=P, n_tokens=5, vocab=100, dim=16, scale=1.0, dtable=P,
                  table_dtype=zs.ZERO_F16, stride=16, workspace=P, workspace_bytes=1 << 20)


@pytest.mark.parametrize("changes, word", [
    (dict(dout=None), "dout"), (dict(dout=P + 1), "aligned"), (dict(dtype=0), "dtype"), (dict(table_dtype=9), "dtype"),
    (dict(table_dtype=zs.ZERO_BF16), "dtable"), (dict(dtype=zs.ZERO_F32), "dtable"), (dict(tokens=None), "tokens"),
    (dict(tokens=P + 4), "aligned"), (dict(vocab=0), "vocab"), (dict(dim=0), "dim"), (dict(scale=NAN), "scale"),
    (dict(dtable=None), "table"), (dict(dtable=P + 1), "aligned"), (dict(stride=15), "overlap"),
    (dict(n_tokens=(1 << 28) + 1), "n_tokens"), (dict(scale=1e39), "scale"), (dict(workspace=None), "workspace"),
    (dict(workspace_bytes=64), "needs"),
    (dict(workspace=P + 64), "256"),
])
def test_embedding_grad_refuses(changes, word):
    refused(zs.lib().zero_embedding_grad(made(zs.EmbeddingGradArgs, EMBED_GRAD, changes), None), word)


def test_embedding_grad_without_tokens_onto_another_gradient_does_nothing():
    assert zs.lib().zero_embedding_grad(None, None) == zs.ZERO_EINVAL
    none = dict(n_tokens=0, accumulate=1, dout=None, tokens=None, workspace=None)
    assert zs.lib().zero_embedding_grad(made(zs.EmbeddingGradArgs, EMBED_GRAD, none), None) == zs.ZERO_OK


# x, residual, gain, dtype, n_rows, dim, eps, h, out, rstd, codes, scales
NORM = [P, P, P, zs.ZERO_BF16, 3, 16, 1e-6, P, P, P, P, P, None]


@pytest.mark.parametrize("at, bad, word", [
    (0, None, "x"), (0, P + 1, "aligned"), (1, None, "together"), (1, P + 1, "aligned"), (2, None, "gain"),
    (3, 0, "dtype"), (4, 1 << 62, "overflows"), (5, 0, "dim"), (5, (1 << 14) + 1, "dim"), (6, NAN, "eps"),
    (6, -1.0, "eps"), (7, None, "together"), (8, None, "out"), (9, P + 2, "aligned"), (10, None, "together"),
    (11, None, "together"), (11, P + 2, "aligned"),
])
def test_norm_refuses(at, bad, word):
    refused(zs.lib().zero_rms_norm(*[bad if i == at else x for i, x in enumerate(NORM)]), word)


# codes, scales, rstd, gain, dtype, n_rows, dim, out
RESTORE = [P, P, P, P, zs.ZERO_F32, 3, 16, P, None]


@pytest.mark.parametrize("at, bad, word", [
    (0, None, "codes"), (1, None, "scales"), (1, P + 2, "aligned"), (2, None, "rstd"), (3, None, "gain"), (3, P + 2, "aligned"),
    (4, 7, "dtype"), (6, 0, "dim"), (7, None, "out"), (7, P + 2, "aligned"),
])
def test_restore_refuses(at, bad, word):
    refused(zs.lib().zero_rms_norm_restore(*[bad if i == at else x for i, x in enumerate(RESTORE)]), word)


BACKWARD = dict(dy=P, gain=P, h=P, rstd=P, upstream=P, dtype=zs.ZERO_F16, n_rows=3, dim=16, dx=P, dgain=P, workspace=P,
                workspace_bytes=1 << 20)


@pytest.mark.parametrize("changes, word", [
    (dict(dy=None), "dy"), (dict(dy=P + 1), "aligned"), (dict(gain=None), "gain"), (dict(h=None), "either"),
    (dict(codes=P), "together"), (dict(codes=P, scales=P), "either"), (dict(scales=P), "together"),
    (dict(h=None, codes=P, scales=P + 2), "aligned"), (dict(rstd=None), "rstd"), (dict(upstream=P + 1), "aligned"),
    (dict(dtype=0), "dtype"), (dict(dim=0), "dim"), (dict(dx=None), "dx"), (dict(dgain=None), "dgain"),
    (dict(dgain=P + 1), "aligned"), (dict(workspace=None), "workspace"), (dict(workspace_bytes=100), "needs"),
    (dict(workspace=P + 64), "256"),
])
def test_norm_backward_refuses(changes, word):
    refused(zs.lib().zero_rms_norm_backward(made(zs.RmsNormBackwardArgs, BACKWARD, changes), None), word)


def test_norm_of_no_rows_does_nothing():
    L = zs.lib()
    assert L.zero_rms_norm_backward(None, None) == zs.ZERO_EINVAL
    assert L.zero_rms_norm(None, None, None, zs.ZERO_F32, 0, 16, 1e-6, None, None, None, None, None, None) == zs.ZERO_OK
    assert L.zero_rms_norm_restore(None, None, None, None, zs.ZERO_F32, 0, 16, None, None) == zs.ZERO_OK


HEAD = dict(hidden=P, weight=P, dtype=zs.ZERO_BF16, n_rows=5, vocab=300, dim=64, hidden_stride=64, weight_stride=64,
            targets=P, row_weight=P, divisor=1.0, temperature=1.0, grad_scale=1.0, stats=P, logp=P, dhidden=P, dweight=P,
            dhidden_stride=64, dweight_stride=64, piece_rows=128, workspace=P, workspace_bytes=1 << 24)


@pytest.mark.parametrize("changes, word", [
    (dict(hidden=None), "hidden"), (dict(hidden=P + 8), "hidden"), (dict(weight=None), "weight"), (dict(weight=P + 2), "weight"),
    (dict(dtype=zs.ZERO_F32), "dtype"), (dict(dtype=0), "dtype"), (dict(n_rows=1 << 31), "n_rows"), (dict(vocab=0), "vocab"),
    (dict(vocab=(1 << 20) + 1), "vocab"), (dict(dim=0), "dim"), (dict(dim=60), "dim"), (dict(dim=(1 << 15) + 8), "dim"),
    (dict(hidden_stride=56), "stride"), (dict(weight_stride=68), "weight"), (dict(weight_stride=1 << 23), "stride"),
    (dict(targets=None), "targets"), (dict(targets=P + 4), "targets"), (dict(row_weight=P + 2), "misaligned"),
    (dict(divisor=0.0), "divisor"), (dict(divisor=NAN), "non-finite"), (dict(temperature=0.0), "temperature"),
    (dict(temperature=1e-60), "temperature"), (dict(grad_scale=INF), "non-finite"), (dict(stats=None), "stats"),
    (dict(logp=None), "logp"), (dict(dhidden=P + 2), "dhidden"), (dict(dhidden_stride=32), "stride"),
    (dict(dweight=P + 4), "dweight"), (dict(dweight_stride=60), "dweight"), (dict(piece_rows=0), "piece_rows"),
    (dict(piece_rows=20000), "piece_rows"), (dict(workspace=None), "workspace"), (dict(workspace_bytes=1000), "needs"),
    (dict(workspace=P + 64), "256"),
])
def test_linear_cross_entropy_refuses(changes, word):
    refused(zs.lib().zero_linear_cross_entropy(made(zs.LinearCrossEntropyArgs, HEAD, changes), None), word)


def test_workspace_sizes():
    L = zs.lib()
    assert L.zero_linear_cross_entropy(None, None) == zs.ZERO_EINVAL
    for fn, args in ((L.zero_embedding_workspace_bytes, (5, 8)), (L.zero_rms_norm_workspace_bytes, (5, 8)),
                     (L.zero_linear_cross_entropy_workspace_bytes, (5, 100, 8, 128, 1))):
        assert fn(*args, None) == zs.ZERO_EINVAL
        assert size(fn, *args) > 0
    assert L.zero_embedding_workspace_bytes(1 << 31, 8, np.zeros(1, np.uint64).ctypes.data) == zs.ZERO_ERANGE
    for bad in ((5, 0, 8, 128, 1), (5, 100, 9, 128, 1), (5, 100, 8, 0, 1)):
        assert L.zero_linear_cross_entropy_workspace_bytes(*bad, np.zeros(1, np.uint64).ctypes.data) == zs.ZERO_EINVAL
    # of 65,536 rows with 128,000 logits: bounded by the piece, not by the rows
    head = L.zero_linear_cross_entropy_workspace_bytes
    whole, piece = 65_536 * 128_000 * 4, size(head, 65_536, 128_000, 4096, 4096, 1)
    assert piece < whole / 6
    # one piece needs no fp32 sums of the weights' gradient, scores no probabilities
    assert size(head, 4096, 128_000, 4096, 4096, 1) < piece - 128_000 * 4096 * 4 + (1 << 20)
    assert size(head, 65_536, 128_000, 4096, 4096, 0) < 100 << 20
    # fewer rows than a workspace was made for fit in it
    for grad in (0, 1):
        last = 0
        for n in (0, 1, 15, 16, 17, 255, 256, 257, 1000, 4096):
            now = size(head, n, 50_001, 1000, 4096, grad)
            assert now >= last, (n, grad)
            last = now


@pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc not found")
@pytest.mark.parametrize("source", ["embed.hip", "norm.hip", "head.hip"])
def test_kernels_keep_to_registers(source):
    """No kernel spills to scratch memory, and none uses packed fp32 arithmetic or an fma that
    rounds straight to 16 bits."""
    from zero_sharded_optimizer_owned_amd.build import CSRC, HIPCC_FLAGS, INCLUDE

    flags = [f for f in HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    res = subprocess.run(["hipcc", *flags, "-I", INCLUDE, "--cuda-device-only", "-S", os.path.join(CSRC, source), "-o", "-"],
                         capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stderr[-2000:]
    sizes = [int(x) for x in re.findall(r"; ScratchSize: (\d+)", res.stdout)]
    assert sizes and max(sizes) == 0, sizes
    assert not re.search(r"v_pk_(add|mul|fma)_f32|v_fma_mix|v_mad_mix", res.stdout)
    if source == "head.hip":  # products on the matrix cores, tiles loaded straight into LDS
        assert "v_mfma_f32_16x16x32_bf16" in res.stdout and "v_mfma_f32_16x16x32_f16" in res.stdout
        assert "ds_read_b64_tr_b16" in res.stdout and re.search(r"buffer_load_dwordx4 .* lds", res.stdout)


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x, t, f = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64), torch.zeros(2)
    for call in (lambda: zs.zero_embedding(x, t, x), lambda: zs.zero_rms_norm(x, x[0], x),
                 lambda: zs.zero_embedding_grad(x, t, x, workspace=f),
                 lambda: zs.zero_rms_norm_backward(x, x[0], f, x, x[0], workspace=f, h=x),
                 lambda: zs.zero_linear_cross_entropy(x.half(), x.half(), t, divisor=1.0, stats=f, logp=f, workspace=f)):
        with pytest.raises((ValueError, RuntimeError)):
            call()
