"""The 8-bit step's piece table and the refusals of the 8-bit step and the losses,
on the CPU: host calls and argument checks only, nothing is launched."""
import ctypes as ct
import functools
import os
import random
import re
import shutil
import subprocess

import numpy as np
import pytest

import oracle
import zero_sharded_optimizer_owned_amd as zs

M = zs.ZERO_PIECE // 8


def covered(pieces, masks, end):
    """The flat elements that the table marks as real, in order."""
    out = []
    for p in pieces:
        flat, n = int(p["flat"]), int(p["len"])
        if int(p["mask"]) == zs.ZERO_PIECE_WHOLE:
            out += range(flat, flat + n)
        else:
            bits = np.unpackbits(masks[int(p["mask"])], bitorder="little")
            assert not bits[n:].any()
            out += [flat + int(i) for i in np.nonzero(bits)[0]]
    return out


def test_piece_table_marks_the_real_elements_once_in_order():
    rnd = random.Random(4)
    for _ in range(300):
        numels = [rnd.randrange(1, rnd.choice([4, 100, 9000])) for _ in range(rnd.randrange(1, 40))]
        ranks, align = rnd.randrange(1, 9), rnd.choice([1, 8, 64, 128])
        off, total, b, e = zs.zero_shard_layout(numels, ranks, align)
        for r in range(ranks):
            begin, end = int(b[r]), int(e[r])
            pieces, masks = zs.zero_piece_table(numels, off, begin, end)
            want = [f for s, t in oracle.real_ranges(numels, [int(x) for x in off], begin, end) for f in range(s, t)]
            assert covered(pieces, masks, end) == want
            base = begin // zs.ZERO_QBLOCK * zs.ZERO_QBLOCK
            flats = [int(p["flat"]) for p in pieces]
            assert flats == sorted(set(flats))
            for p in pieces:
                flat, n = int(p["flat"]), int(p["len"])
                assert flat >= base and flat % zs.ZERO_QBLOCK == 0 and 1 <= n <= zs.ZERO_PIECE
                assert flat // zs.ZERO_PIECE == (flat + n - 1) // zs.ZERO_PIECE  # within one window
                assert int(p["mask"]) != zs.ZERO_PIECE_WHOLE or n % 8 == 0
            assert sorted(int(p["mask"]) for p in pieces if int(p["mask"]) != zs.ZERO_PIECE_WHOLE) == list(
                range(len(masks)))


def test_piece_table_of_an_unpadded_run_is_whole_but_for_its_end():
    off, total, b, e = zs.zero_shard_layout([10_000_000_000], 7, 64)
    pieces, masks = zs.zero_piece_table([10_000_000_000], off, int(b[3]), int(b[3]) + 100_000)
    assert len(masks) <= 2 and len(pieces) in (49, 50)
    assert all(int(p["mask"]) == zs.ZERO_PIECE_WHOLE for p in pieces[1:-1])


def test_piece_table_empty_owner_capacity_and_errors():
    off, total, b, e = zs.zero_shard_layout([100, 50], 1, 8)
    pieces, masks = zs.zero_piece_table([100, 50], off, 50, 50)
    assert pieces.size == 0 and masks.shape == (0, M)
    n = np.array([100, 5000], dtype=np.uint64)
    o = np.array([0, 104], dtype=np.uint64)
    L, cnt, nm = zs.lib(), np.zeros(1, np.uint64), np.zeros(1, np.uint64)
    out, mk = np.zeros(1, dtype=zs.PIECE_DTYPE), np.zeros((1, M), np.uint8)
    args = (n.ctypes.data, o.ctypes.data, 2, 0, 5104)
    assert L.zero_piece_table(*args, out.ctypes.data, 1, mk.ctypes.data, 1, cnt.ctypes.data,
                              nm.ctypes.data) == zs.ZERO_ERANGE
    assert int(cnt[0]) == 3 and int(nm[0]) == 2
    assert L.zero_piece_table(n.ctypes.data, o.ctypes.data, 2, 9, 5, None, 0, None, 0, cnt.ctypes.data,
                              nm.ctypes.data) == zs.ZERO_EINVAL
    bad = np.array([0, 90], dtype=np.uint64)  # overlaps
    assert L.zero_piece_table(n.ctypes.data, bad.ctypes.data, 2, 0, 5104, None, 0, None, 0, cnt.ctypes.data,
                              nm.ctypes.data) == zs.ZERO_EINVAL
    zero = np.array([0, 5], dtype=np.uint64)
    assert L.zero_piece_table(zero.ctypes.data, o.ctypes.data, 2, 0, 50, None, 0, None, 0, cnt.ctypes.data,
                              nm.ctypes.data) == zs.ZERO_EINVAL
    assert L.zero_piece_table(*args, None, 0, None, 0, None, nm.ctypes.data) == zs.ZERO_EINVAL
    with pytest.raises(ValueError):
        zs.zero_piece_table([1, 2], [0], 0, 3)


def refused(rc, word):
    assert rc == zs.ZERO_EINVAL
    assert word in zs.lib().zero_last_error().decode(), zs.lib().zero_last_error()


def adam8(**changes):
    """Arguments that pass every check (none of the addresses is looked at on the host)."""
    a = zs.Adam8Args()
    a.pieces, a.n_pieces, a.begin, a.end, a.local_base = 4096, 1, 300, 400, 256
    a.reduced_g = a.master = a.exp_avg8 = a.exp_rms8 = a.exp_avg_scale = a.exp_rms_scale = 4096
    a.step, a.lr, a.beta1, a.beta2, a.eps, a.clip_coef = 1, 1e-3, 0.9, 0.99, 1e-8, 1.0
    for k, v in changes.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("changes, word", [
    (dict(step=0), "step"), (dict(begin=500), "begin > end"), (dict(pieces=None), "pieces"),
    (dict(n_masks=2), "masks"), (dict(local_base=128 + 8), "local_base"), (dict(local_base=384), "local_base"),
    (dict(exp_avg8=None), "state"), (dict(exp_rms_scale=None), "state"), (dict(exp_rms8=4097), "aligned"),
    (dict(reduced_g=4100), "reduced_g"), (dict(master=None), "master"), (dict(master=4104), "aligned"),
    (dict(param_dtype=zs.ZERO_F32), "param_dtype"), (dict(param_dtype=zs.ZERO_F16), "param16"),
    (dict(param_dtype=zs.ZERO_BF16, param16=4096, param_base=4), "param_base"),
    (dict(lr=float("nan")), "non-finite"), (dict(lr=-1.0), "lr"), (dict(beta1=1.0), "betas"),
    (dict(beta2=-0.1), "betas"), (dict(clip_coef=-1.0), "clip_coef"),
    (dict(reduced_g=None), "R = 0"), (dict(reduced_g=None, R=2), "rank_grads"),
    (dict(reduced_g=None, R=zs.ZERO_MAX_RANKS + 1), "outside"),
])
def test_adam8_step_refuses(changes, word):
    refused(zs.lib().zero_adam8_step(ct.byref(adam8(**changes)), None), word)


@pytest.mark.parametrize("changes, word", [
    (dict(grad_dtype=9), "dtype"), (dict(grad_base=4), "grad_base"), (dict(grad_base=304), "grad_base"),
    (dict(divisor=0.0), "divisor"), (dict(divisor=float("inf")), "divisor"),
])
def test_adam8_step_refuses_rank_gradients(changes, word):
    ranks = (ct.c_void_p * 2)(4096, 4096)
    base = dict(reduced_g=None, R=2, rank_grads=ct.cast(ranks, ct.c_void_p), grad_dtype=zs.ZERO_F16, divisor=2.0)
    refused(zs.lib().zero_adam8_step(ct.byref(adam8(**{**base, **changes})), None), word)
    for bad, why in ((0, "NULL"), (4098, "aligned")):
        ranks[1] = bad
        refused(zs.lib().zero_adam8_step(ct.byref(adam8(**base)), None), why)


def test_adam8_step_without_work_does_nothing():
    assert zs.lib().zero_adam8_step(None, None) == zs.ZERO_EINVAL
    for none in (dict(n_pieces=0), dict(begin=400)):
        assert zs.lib().zero_adam8_step(ct.byref(adam8(**none)), None) == zs.ZERO_OK


def test_moments8_refuse():
    L, p = zs.lib(), 4096
    for fn, name in ((L.zero_moments8_pack, "pack"), (L.zero_moments8_unpack, "unpack")):
        good = [p, 1, None, 0, 300, 400, 256, p, p, p, p, p, p, None]
        assert fn(*good[:1], 0, *good[2:]) == zs.ZERO_OK  # no pieces: no work
        for at, bad, word in ((0, None, "pieces"), (3, 1, "masks"), (4, 500, "begin"), (6, 130, "local_base")):
            refused(fn(*[bad if i == at else x for i, x in enumerate(good)]), word)
        for at in range(7, 13):
            for bad in (None, p + 4):
                rc = fn(*[bad if i == at else x for i, x in enumerate(good)])
                assert rc == zs.ZERO_EINVAL, (name, at, bad)


def test_token_logprobs_refuses():
    L, p, nan = zs.lib(), 4096, float("nan")
    good = [p, zs.ZERO_BF16, 3, 10, 10, p, 1.0, p, None]
    for at, bad, word in ((1, 0, "dtype"), (3, 0, "vocab"), (4, 9, "overlap"), (6, 0.0, "temperature"),
                          (6, nan, "temperature"), (6, 1e-60, "temperature"), (0, None, "logits"), (5, None, "targets"),
                          (0, p + 1, "aligned"), (5, p + 4, "aligned"), (7, None, "logp"), (7, p + 2, "logp"),
                          (2, 2 ** 62, "overflows")):
        refused(L.zero_token_logprobs(*[bad if i == at else x for i, x in enumerate(good)]), word)
    assert L.zero_token_logprobs(None, zs.ZERO_F32, 0, 10, 10, None, 1.0, None, None) == zs.ZERO_OK


def policy(**changes):
    a = zs.PolicyArgs()
    a.logits = a.targets = a.old_logp = a.ref_logp = a.advantage = a.weight = a.stats = a.logp = a.dlogits = 4096
    a.workspace, a.workspace_bytes = 4096, 1 << 20
    a.dtype, a.n_rows, a.vocab, a.row_stride, a.dlogits_stride = zs.ZERO_F16, 5, 100, 100, 100
    a.divisor, a.clip_low, a.clip_high, a.kl_coef, a.temperature, a.grad_scale = 1.0, 0.2, 0.2, 0.1, 1.0, 1.0
    for k, v in changes.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("changes, word", [
    (dict(dtype=0), "dtype"), (dict(vocab=0), "vocab"), (dict(row_stride=99), "overlap"),
    (dict(temperature=-1.0), "temperature"), (dict(logits=None), "logits"), (dict(targets=None), "targets"),
    (dict(divisor=0.0), "divisor"), (dict(divisor=float("nan")), "non-finite"), (dict(clip_low=1.5), "clip_low"),
    (dict(clip_high=-0.1), "clip_high"), (dict(kl_coef=-1.0), "kl_coef"), (dict(ref_logp=None), "ref_logp"),
    (dict(grad_scale=float("inf")), "non-finite"), (dict(dlogits=4097), "dlogits"), (dict(dlogits_stride=50), "dlogits"),
    (dict(stats=None), "stats"), (dict(old_logp=None), "old_logp"), (dict(advantage=None), "advantage"),
    (dict(logp=None), "logp"), (dict(weight=4098), "misaligned"), (dict(workspace=None), "workspace"),
    (dict(workspace_bytes=64), "workspace needs"), (dict(workspace=4096 + 64), "256"),
])
def test_policy_loss_refuses(changes, word):
    refused(zs.lib().zero_policy_loss(ct.byref(policy(**changes)), None), word)


def preference(**changes):
    a = zs.PreferenceArgs()
    a.logits = a.targets = a.seq_begin = a.ref_logp = a.stats = a.logp = a.seq_logp = a.reward = a.dlogits = 4096
    a.workspace, a.workspace_bytes = 4096, 1 << 20
    a.dtype, a.n_rows, a.vocab, a.row_stride, a.dlogits_stride, a.n_pairs = zs.ZERO_F32, 5, 100, 100, 100, 2
    a.beta, a.temperature, a.grad_scale = 0.1, 1.0, 1.0
    for k, v in changes.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("changes, word", [
    (dict(dtype=7), "dtype"), (dict(row_stride=1), "overlap"), (dict(temperature=0.0), "temperature"),
    (dict(beta=0.0), "beta"), (dict(beta=float("nan")), "non-finite"), (dict(label_smoothing=0.6), "label_smoothing"),
    (dict(label_smoothing=-0.1), "label_smoothing"), (dict(n_pairs=0), "n_pairs"), (dict(dlogits=4098), "dlogits"),
    (dict(seq_begin=None), "seq_begin"), (dict(ref_logp=None), "ref_logp"), (dict(reward=None), "reward"),
    (dict(seq_begin=4100), "misaligned"), (dict(logp=None), "logp"), (dict(workspace=None), "workspace"),
    (dict(workspace_bytes=100), "workspace needs"),
])
def test_preference_loss_refuses(changes, word):
    refused(zs.lib().zero_preference_loss(ct.byref(preference(**changes)), None), word)


def test_workspace_sizes_cover_every_row():
    L, b = zs.lib(), np.zeros(1, np.uint64)
    for n in (0, 1, 1000, 10 ** 9):
        assert L.zero_policy_workspace_bytes(n, b.ctypes.data) == 0 and int(b[0]) >= 24 * n
        assert L.zero_preference_workspace_bytes(n, 3, b.ctypes.data) == 0 and int(b[0]) >= 24 * n + 48
    assert L.zero_policy_workspace_bytes(1, None) == zs.ZERO_EINVAL
    assert L.zero_preference_workspace_bytes(1, 1, None) == zs.ZERO_EINVAL
    assert L.zero_policy_workspace_bytes(2 ** 60, b.ctypes.data) == zs.ZERO_ERANGE


def test_binding_refuses_host_tensors_and_shapes():
    torch = pytest.importorskip("torch")
    x, t, o = torch.zeros(3, 8), torch.zeros(3, dtype=torch.int64), torch.zeros(3)
    with pytest.raises(ValueError):
        zs.zero_token_logprobs(x, t, o)  # not on a device
    with pytest.raises(TypeError):
        zs.zero_token_logprobs(x.double(), t, o)
    with pytest.raises(ValueError):
        zs.zero_token_logprobs(x[0], t, o)
    with pytest.raises(ValueError):
        zs.zero_preference_loss(x, t, torch.zeros(2, dtype=torch.int64), ref_logp=o, stats=o, logp=o, seq_logp=o,
                                reward=o, workspace=o)


ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@functools.lru_cache(maxsize=None)
def _device_asm(source: str) -> str:
    """gfx950 assembly of one of the library's HIP sources, built with its flags."""
    from zero_sharded_optimizer_owned_amd.build import CSRC, HIPCC_FLAGS, INCLUDE

    flags = [f for f in HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    res = subprocess.run(["hipcc", *flags, "-I", INCLUDE, "--cuda-device-only", "-S",
                          os.path.join(CSRC, source), "-o", "-"], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
    return res.stdout


@pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc not found")
@pytest.mark.parametrize("source", ["step8.hip", "loss.hip"])
def test_kernels_keep_to_registers(source):
    """No kernel spills to scratch memory (rows and batches of loads live in registers), and
    none uses packed fp32 arithmetic or an fma that rounds straight to 16 bits."""
    asm = _device_asm(source)
    sizes = [int(x) for x in re.findall(r"; ScratchSize: (\d+)", asm)]
    assert sizes and max(sizes) == 0, sizes
    assert not re.search(r"v_pk_(add|mul|fma)_f32|v_fma_mix|v_mad_mix", asm)


@pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc not found")
def test_codes_use_the_hardware_conversions():
    asm = _device_asm("step8.hip")
    assert "v_cvt_pk_fp8_f32" in asm and "v_cvt_pk_f32_fp8" in asm


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the ROCm headers not found")
def test_piece_table_under_sanitizers(tmp_path):
    """zero_piece_table over random layouts, built with AddressSanitizer and
    UndefinedBehaviorSanitizer: tables of exactly the counted size, and short ones."""
    exe = str(tmp_path / "piece_driver")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-static-libasan", "-I", os.path.join(ROOT, "include"), "-I", "/opt/rocm/include",
           "-D__HIP_PLATFORM_AMD__", os.path.join(ROOT, "tests", "sanitize", "piece_driver.cpp"),
           os.path.join(ROOT, "zero_sharded_optimizer_owned_amd", "csrc", "host.cpp"), "-o", exe]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0 and "sanitize" in res.stderr and ("cannot find" in res.stderr or "unrecognized" in res.stderr):
        pytest.skip("sanitizer runtime not available: " + res.stderr[-300:])
    assert res.returncode == 0, res.stderr[-3000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=600,
                         env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert run.returncode == 0 and "clean" in run.stdout, run.stdout[-2000:] + run.stderr[-4000:]
