"""The owner step with 8-bit moments against its formula in 64 bits, on the same
decoded state.

Tolerances.  u = 2^-24 is half an fp32 step, relative.  The rank mean is formed
as zero_reduce_owned forms it (checked bit for bit), so the gradient is taken
as the kernel's.  With a = beta1 |m0| + (1 - beta1) |g| and b = beta2 r0^2 +
(1 - beta2) g^2 (no cancellation in b):
  * clip, the two decodings and the fma leave |dm| <= 6 u a and |dr| <= 6 u r;
  * denom and the quotient add 6 u, the product with the step size and the last
    fma 3 u: |dw| <= 3 u |w| + 20 u * (lr / bc1) * a / denom;
  * a scale is a maximum over 448: 8 u of the block's largest a / 448 (or r / 448);
  * a code is the nearest e4m3 value of x / scale: half a step, 2^-4 |x|, or
    2^-10 scale below the normal range, plus 2^-18 |x| for x's and the scale's
    own fp32 errors; a root above zero takes at least the code 2^-9.
"""
import numpy as np
import pytest

import oracle
import synth
from helpers import BF16, F16, F32, assert_bits_equal, from_dev, gen, to_dev, torch_dtype

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import zero_sharded_optimizer_owned_amd as zs  # noqa: E402

DEV = "cuda"
Q = zs.ZERO_QBLOCK
U = 2.0 ** -24
HP = dict(lr=1e-3, beta1=0.8, beta2=0.999, eps=1e-8, weight_decay=3e-7, adamw=True)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    zs.lib()
    yield
    torch.cuda.synchronize()


def make_shard(numels, ranks, owner, align, seed=1, moments=True):
    """A shard with random state; padding of master and param16 holds a sentinel."""
    sh = zs.OwnerShard8(numels, ranks, owner, align=align, device=DEV)
    sh.alloc_state()
    n = sh.master.numel()
    sh.master.copy_(to_dev(gen(seed, synth.STREAM_MASTER, n, synth.DIST_NORMAL, 0.02, F32), F32))
    if moments:
        m = to_dev(gen(seed, synth.STREAM_EXP_AVG, n, synth.DIST_NORMAL, 5e-4, F32), F32)
        v = to_dev(gen(seed, synth.STREAM_EXP_AVG_SQ, n, synth.DIST_SQUARE, 4e-4, F32), F32)
        sh.pack_moments(m, v)
    return sh


def real_mask(sh):
    off, _, owners = oracle.layout(list(sh.numels), sh.ranks, sh.align)
    mask = np.zeros(sh.blocks * Q, dtype=bool)
    for b, e in oracle.real_ranges(sh.numels, off, sh.begin, sh.end):
        mask[b - sh.local_base:e - sh.local_base] = True
    return mask


def host_state(sh):
    """master, codes' values and scales as float64 / numpy."""
    val = lambda c: c.float().cpu().numpy().astype(np.float64)
    return dict(w=sh.master.cpu().numpy().astype(np.float64), m8=val(sh.exp_avg8), r8=val(sh.exp_rms8),
                ms=sh.exp_avg_scale.cpu().numpy().astype(np.float64),
                rs=sh.exp_rms_scale.cpu().numpy().astype(np.float64))


def rank_buffers(sh, R, code, base, seed=2, scale=1e-3, poison=True):
    """Rank gradients from flat index `base`; padding holds NaN (it must not be looked at)."""
    n = sh.blocks * Q + sh.local_base - base
    out = []
    mask = np.zeros(n, dtype=bool)
    mask[sh.local_base - base:] = real_mask(sh)
    for r in range(R):
        g = to_dev(gen(seed, synth.STREAM_GRAD, n, synth.DIST_NORMAL, scale, code, rank=r), code)
        if poison:
            g[torch.from_numpy(~mask).to(DEV)] = float("nan")
        out.append(g)
    return out


def check_step(sh, before, g, hp, step, clip=1.0, p16=None, p_before=None, what=""):
    """The state after a step against the formula in 64 bits; g the fp32 mean gradient (owner-local, numpy)."""
    after, real = host_state(sh), real_mask(sh)
    spread = lambda s: np.repeat(s, Q)
    m0, r0 = before["m8"] * spread(before["ms"]), before["r8"] * spread(before["rs"])
    w0 = before["w"]
    g = np.where(real, g.astype(np.float64), 0.0) * np.float64(np.float32(clip))
    if not hp["adamw"]:
        g = g + hp["weight_decay"] * w0 * real
    b1, b2 = hp["beta1"], hp["beta2"]
    a = (b1 * np.abs(m0) + (1 - b1) * np.abs(g)) * real
    m = (b1 * m0 + (1 - b1) * g) * real
    r = np.sqrt(b2 * r0 ** 2 + (1 - b2) * g ** 2) * real
    denom = r / np.sqrt(1 - b2 ** step) + hp["eps"]
    size = hp["lr"] / (1 - b1 ** step)
    decay = 1 - hp["lr"] * hp["weight_decay"] if hp["adamw"] else 1.0
    with np.errstate(divide="ignore", invalid="ignore"):
        w = np.where(real, w0 * decay - size * m / denom, w0)
        tol = np.where(real, 3 * U * np.abs(w0) + 20 * U * size * a / denom + 1e-30, 0.0)
    bad = np.nonzero(~(np.abs(after["w"] - w) <= tol))[0]
    assert bad.size == 0, f"{what}: master {bad.size} off, first {bad[:4]}: {after['w'][bad[:4]]} vs {w[bad[:4]]}"
    for x, amp, codes, scale, root in ((m, a, after["m8"], after["ms"], False), (r, r, after["r8"], after["rs"], True)):
        top = np.abs(x).reshape(-1, Q).max(1)
        amp_top = amp.reshape(-1, Q).max(1)
        live = top >= 2.0 ** -100
        touched = real.reshape(-1, Q).any(1)
        got = scale[touched]
        assert np.all(np.abs(got - np.where(live, top / 448, 0.0)[touched]) <= 8 * U * amp_top[touched] / 448), what
        value, s = codes * spread(scale), spread(np.where(live, top / 448, 0.0))
        half = np.maximum(np.abs(x) * 2.0 ** -4, s * (2.0 ** -9 if root else 2.0 ** -10))
        ok = np.abs(value - x) <= half + 2.0 ** -18 * np.abs(x) + 8 * U * amp
        assert np.all(ok[real]), f"{what}: codes off at {np.nonzero(real & ~ok)[0][:4]}"
        assert np.all(codes[~real] == 0) or not touched.all(), what
        if root:
            assert np.all((codes > 0)[real & (x > 0) & np.repeat(live, Q)]), f"{what}: a positive root became zero"
    # master outside the real elements is untouched, bit for bit
    assert np.array_equal(after["w"][~real], before["w"][~real]), what
    if p16 is not None:
        code = F16 if p16.dtype == torch.float16 else BF16
        got, idx = from_dev(p16), np.nonzero(real)[0]
        assert_bits_equal(got[idx], oracle.encode16(sh.master.cpu().numpy()[idx], code), what + " copy")
        keep = np.ones(got.size, dtype=bool)
        keep[idx] = False
        assert np.array_equal(got[keep], p_before[keep]), what + ": copy written outside the real elements"


LAYOUTS = [
    ([1000, 37, 5003], 4, 1, 64),            # cuts inside tensors, padding
    ([1000, 37, 5003], 4, 3, 64),            # the ragged end
    ([10_000], 3, 1, 1),                     # one unpadded run, both ends off any boundary
    ([1] * 700, 2, 1, 8),                    # one element in each vector
    ([5, 300, 3, 129, 128, 127], 1, 0, 1),   # tensors meeting inside blocks, no padding
    ([100] * 300, 2, 0, 64),                 # short padded tensors
    ([4096 * 16], 2, 1, 64),                 # whole pieces only
    ([7], 4, 1, 1),                          # owner of one element
]


@pytest.mark.parametrize("layout", range(len(LAYOUTS)))
@pytest.mark.parametrize("R, gcode, pcode", [(1, F32, None), (2, F16, F16), (3, BF16, BF16), (8, BF16, None),
                                             (5, F32, F16), (16, F16, BF16), (33, F16, F16)])
def test_step_matches_the_formula(layout, R, gcode, pcode):
    numels, ranks, owner, align = LAYOUTS[layout]
    sh = make_shard(numels, ranks, owner, align)
    base = sh.local_base
    grads = rank_buffers(sh, R, gcode, base)
    p16 = None
    if pcode:
        p16 = to_dev(gen(9, synth.STREAM_MASTER, sh.blocks * Q, synth.DIST_NORMAL, 1.0, pcode), pcode)
    before, p_before = host_state(sh), from_dev(p16) if pcode else None
    sh.adam_step(step=7, hyper=HP, rank_grads=grads, grad_base=base, divisor=float(R), param16=p16, param_base=base)
    torch.cuda.synchronize()
    g = oracle.reduce([from_dev(x) for x in grads], gcode, float(R))
    check_step(sh, before, g, HP, 7, p16=p16, p_before=p_before, what=f"layout {layout}, R {R}")


@pytest.mark.parametrize("hp, step, clip", [
    (dict(HP, adamw=False, weight_decay=0.1), 1, 1.0), (dict(HP, weight_decay=0.1), 1, 0.25),
    (dict(HP, beta1=0.0, beta2=0.0), 3, 1.0), (dict(HP, beta1=0.9, beta2=0.95, eps=1e-5), 2 ** 40, 1.0),
    (dict(HP, lr=0.0), 5, 1.0), (HP, 5, 0.0),
])
def test_hyperparameters_and_stored_gradient(hp, step, clip):
    sh = make_shard([5003, 70, 20_000], 2, 1, 64)
    g = gen(3, synth.STREAM_GRAD, sh.blocks * Q, synth.DIST_NORMAL, 1e-3, F32)
    before = host_state(sh)
    sh.adam_step(step=step, hyper=hp, reduced_g=to_dev(g, F32), clip_coef=clip)
    torch.cuda.synchronize()
    check_step(sh, before, g, hp, step, clip=clip, what=str((hp, step, clip)))


def state_bits(sh):
    return [x.view(torch.uint8).cpu().numpy().copy() for x in (sh.master, sh.exp_avg8, sh.exp_avg_scale, sh.exp_rms8,
                                                                sh.exp_rms_scale)]


def copy_state(src, dst):
    for k in zs.OwnerShard8._SAVED:
        getattr(dst, k).copy_(getattr(src, k))


@pytest.mark.parametrize("code, R, divisor", [(F16, 4, 4.0), (BF16, 3, 3.0), (F32, 9, 9.0 * 65536)])
def test_rank_gradients_equal_the_stored_reduction_bit_for_bit(code, R, divisor):
    numels = [1000, 37, 5003, 9000]
    a, b = (make_shard(numels, 2, 1, 64) for _ in range(2))
    grads = rank_buffers(a, R, code, 0, poison=False)
    g = torch.zeros(a.blocks * Q, dtype=torch.float32, device=DEV)
    zs.zero_reduce_owned(grads, a.begin, a.end - a.begin, divisor, g, out_base=a.local_base)
    a.adam_step(step=2, hyper=HP, rank_grads=grads, divisor=divisor)
    b.adam_step(step=2, hyper=HP, reduced_g=g)
    for x, y in zip(state_bits(a), state_bits(b)):
        assert np.array_equal(x, y)


def test_owners_together_equal_the_unsharded_step_on_whole_blocks():
    """Owners cut at block boundaries give the unsharded state bit for bit."""
    numels, R = [Q * 48 * 4], 4
    whole = make_shard(numels, 1, 0, 1)
    parts = [zs.OwnerShard8(numels, R, r, align=1, device=DEV) for r in range(R)]
    g = to_dev(gen(5, synth.STREAM_GRAD, numels[0], synth.DIST_NORMAL, 1e-3, BF16), BF16)
    for r, sh in enumerate(parts):
        sh.alloc_state()
        for k in zs.OwnerShard8._SAVED:
            src, n = getattr(whole, k), getattr(sh, k).numel()
            getattr(sh, k).copy_(src[r * n:(r + 1) * n])
    whole.adam_step(step=4, hyper=HP, rank_grads=[g])
    for sh in parts:
        sh.adam_step(step=4, hyper=HP, rank_grads=[g])
    for k in zs.OwnerShard8._SAVED:
        bits = lambda t: t.view(torch.uint8).cpu()
        assert torch.equal(bits(getattr(whole, k)), torch.cat([bits(getattr(sh, k)) for sh in parts])), k


def test_flat_indices_beyond_32_bits():
    numels = [20_000_000_001]
    sh = make_shard(numels, 4_000_000, 3_999_998, 1)
    assert sh.begin > 2 ** 34
    grads = rank_buffers(sh, 2, F16, sh.local_base)
    before = host_state(sh)
    sh.adam_step(step=7, hyper=HP, rank_grads=grads, grad_base=sh.local_base, divisor=2.0)
    check_step(sh, before, oracle.reduce([from_dev(x) for x in grads], F16, 2.0), HP, 7)


def test_empty_owner_and_an_empty_table_change_nothing():
    sh = zs.OwnerShard8([3], 8, 0, align=1, device=DEV)
    assert sh.begin == sh.end
    sh.alloc_state()
    sh.master.fill_(5.0)
    sh.adam_step(step=1, hyper=HP, rank_grads=[torch.ones(8, device=DEV)])
    assert sh.checked_step(step=1, hyper=HP, rank_grads=[torch.ones(8, device=DEV)]) == (True, 1.0)
    assert float(sh.master.min()) == 5.0


def test_bad_table_entries_are_skipped():
    """Pieces off the block grid, too long, below the base, or with a mask index
    past the masks are skipped, and elements outside [begin, end) are ignored."""
    sh = make_shard([Q * 64], 1, 0, 1)
    before = state_bits(sh)
    W = zs.ZERO_PIECE_WHOLE
    bad = np.array([(8, 64, W), (0, 4096, W), (0, 128, 0), (128, 128, 7), (Q * 64, 2048, W), (2 ** 63, 2048, W)],
                   dtype=zs.PIECE_DTYPE)
    st = dict(sh._state8(), pieces_dev=zs.chunks_to_device(bad), n_pieces=bad.size, masks_dev=None)
    g = torch.ones(sh.blocks * Q, device=DEV)
    zs.zero_adam8_step(**st, master=sh.master, step=1, reduced_g=g, **HP)
    for x, y in zip(state_bits(sh), before):
        assert np.array_equal(x, y)
    st.update(begin=256, end=300, local_base=128)  # the shard's own table, a narrower range
    st.update(pieces_dev=sh.pieces_dev, n_pieces=sh.pieces.size)
    for k in ("exp_avg8", "exp_rms8", "exp_avg_scale", "exp_rms_scale"):
        st[k] = getattr(sh, k)[(1 if k.endswith("scale") else Q):].clone()  # the views' own memory, 16-byte aligned
    w = sh.master[128:].clone()
    pieces = np.array([(128, 2048 - 128, W)], dtype=zs.PIECE_DTYPE)
    st.update(pieces_dev=zs.chunks_to_device(pieces), n_pieces=1)
    w0 = w.clone()
    zs.zero_adam8_step(**st, master=w, step=1, reduced_g=g[:w.numel()].clone(), **HP)
    changed = (w != w0).cpu().numpy().nonzero()[0]
    assert changed.size and changed.min() >= 128 and changed.max() < 172


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_non_finite_gradient_stays_in_its_block(bad):
    sh = make_shard([Q * 40], 1, 0, 1)
    g = to_dev(gen(3, synth.STREAM_GRAD, Q * 40, synth.DIST_NORMAL, 1e-3, F32), F32)
    g[5 * Q + 17] = bad
    sh.adam_step(step=2, hyper=HP, reduced_g=g)
    fine = torch.isfinite(sh.exp_avg_scale)
    assert not bool(fine[5]) and int((~fine).sum()) == 1
    w = torch.isfinite(sh.master)
    assert int((~w).sum()) == 1 and not bool(w[5 * Q + 17])


def test_zero_gradients_tiny_blocks_and_scales():
    """Blocks of zeros hold zeros, blocks below 2^-100 are dropped, values far
    apart in one block keep what e4m3 holds of them."""
    n = Q * 4
    sh = zs.OwnerShard8([n], 1, 0, align=1, device=DEV)
    sh.alloc_state()
    m, v = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    m[Q:2 * Q] = 1e-35
    v[Q:2 * Q] = 1e-44  # a subnormal; its root is 1e-22
    m[2 * Q], m[2 * Q + 1] = 448.0, -1.0
    v[2 * Q], v[2 * Q + 1] = 1e10, 1e-30  # the smaller root would round to zero
    m[3 * Q:], v[3 * Q:] = 3e38, 3e38
    sh.pack_moments(m, v)
    assert float(sh.exp_avg_scale[0]) == float(sh.exp_rms_scale[0]) == float(sh.exp_avg_scale[1]) == 0.0
    assert float(sh.exp_rms_scale[1]) > 0
    got_m, got_v = torch.full_like(m, -1), torch.full_like(v, -1)
    sh.unpack_moments(got_m, got_v)
    assert float(got_m[0]) == float(got_v[0]) == float(got_m[Q]) == 0.0
    assert float(got_m[2 * Q]) == 448.0 and float(got_m[2 * Q + 1]) == -1.0
    assert float(got_v[2 * Q + 1]) > 0
    assert bool(torch.isfinite(got_m[3 * Q:]).all())
    w = sh.master.clone()
    sh.adam_step(step=1, hyper=dict(HP, eps=1e-8), reduced_g=torch.zeros(n, device=DEV))
    assert torch.equal(sh.master[:Q], w[:Q]) and bool(torch.isfinite(sh.master).all())


@pytest.mark.parametrize("layout", range(len(LAYOUTS)))
def test_pack_and_unpack(layout):
    numels, ranks, owner, align = LAYOUTS[layout]
    sh = make_shard(numels, ranks, owner, align, moments=False)
    real, n = real_mask(sh), sh.blocks * Q
    m = gen(1, synth.STREAM_EXP_AVG, n, synth.DIST_NORMAL, 5e-4, F32)
    v = gen(1, synth.STREAM_EXP_AVG_SQ, n, synth.DIST_SQUARE, 4e-4, F32)
    m[~real] = np.nan  # must not be looked at
    v[~real] = np.nan
    sh.pack_moments(to_dev(m, F32), to_dev(v, F32))
    gm, gv = (torch.full((n,), -3.0, device=DEV) for _ in range(2))
    sh.unpack_moments(gm, gv)
    gm, gv = gm.cpu().numpy().astype(np.float64), gv.cpu().numpy().astype(np.float64)
    assert np.all(gm[~real] == -3.0) and np.all(gv[~real] == -3.0)
    m, r = np.where(real, m, 0.0).astype(np.float64), np.sqrt(np.where(real, v, 0.0).astype(np.float64))
    for x, got, root in ((m, gm, False), (r, np.sqrt(np.abs(gv)), True)):
        s = np.repeat(np.abs(x).reshape(-1, Q).max(1) / 448, Q)
        half = np.maximum(np.abs(x) * 2.0 ** -4, s * (2.0 ** -9 if root else 2.0 ** -10)) + 2.0 ** -18 * np.abs(x)
        assert np.all((np.abs(got - x) <= half)[real])
    # what came out packs back into the same codes
    codes = [x.view(torch.uint8).cpu().numpy().copy() for x in (sh.exp_avg8, sh.exp_rms8)]
    sh.unpack_moments(a := torch.zeros(n, device=DEV), b := torch.zeros(n, device=DEV))
    sh.pack_moments(a, b)
    for x, y in zip(codes, (sh.exp_avg8, sh.exp_rms8)):
        assert np.array_equal(x[real], y.view(torch.uint8).cpu().numpy()[real])


def test_checked_step_skips_clips_and_updates():
    sh = make_shard([5003, 70, 20_000], 2, 1, 64)
    R, scale = 4, 65536.0
    grads = rank_buffers(sh, R, F16, 0, scale=0.2 * scale / 16, poison=False)
    real = np.zeros(sh.padded_total, dtype=bool)
    off, _, _ = oracle.layout(list(sh.numels), 2, 64)
    for b, e in oracle.real_ranges(sh.numels, off, sh.begin, sh.end):
        real[b:e] = True
    for g in grads:
        g[torch.from_numpy(~real[:g.numel()]).to(DEV) if g.numel() <= real.size else
          torch.from_numpy(~np.pad(real, (0, g.numel() - real.size))).to(DEV)] = 0
    g = oracle.reduce([from_dev(x)[sh.local_base:sh.local_base + sh.blocks * Q] for x in grads], F16, R * scale)
    g = np.pad(g, (0, sh.blocks * Q - g.size))
    sumsq = float((g.astype(np.float64) ** 2 * real_mask(sh)).sum())
    for max_norm in (1.0, 0.1):  # the gradient's norm lies between them
        before = host_state(sh)
        updated, coef = sh.checked_step(step=3, hyper=HP, rank_grads=grads, divisor=R * scale, max_norm=max_norm)
        assert updated and abs(coef - min(1.0, max_norm / (sumsq ** 0.5 + 1e-6))) <= 1e-6
        assert (coef < 1) == (max_norm < 1)
        check_step(sh, before, g, HP, 3, clip=coef)
    kept = state_bits(sh)
    grads[1][sh.begin + 3] = float("inf")
    assert sh.checked_step(step=4, hyper=HP, rank_grads=grads, divisor=R * scale) == (False, None)
    for x, y in zip(state_bits(sh), kept):
        assert np.array_equal(x, y)


def test_save_and_load_resume_bit_for_bit(tmp_path):
    a = make_shard([5003, 70, 2000], 2, 1, 64)
    g = to_dev(gen(3, synth.STREAM_GRAD, a.blocks * Q, synth.DIST_NORMAL, 1e-3, F32), F32)
    a.adam_step(step=1, hyper=HP, reduced_g=g)
    a.save(str(tmp_path / "s.npz"), 1)
    b = zs.OwnerShard8([5003, 70, 2000], 2, 1, align=64, device=DEV)
    assert b.load(str(tmp_path / "s.npz")) == 1
    for sh in (a, b):
        sh.adam_step(step=2, hyper=HP, reduced_g=g)
    for x, y in zip(state_bits(a), state_bits(b)):
        assert np.array_equal(x, y)
    with pytest.raises(ValueError):
        zs.OwnerShard8([5003, 70, 2001], 2, 1, align=64, device=DEV).load(str(tmp_path / "s.npz"))


def test_master_exports_through_the_dense_layout():
    sh = make_shard([100, 37, 5003], 2, 1, 64)
    dense = torch.zeros(sh.dense_total, device=DEV)
    sh.to_dense(sh.master, dense)
    back = torch.zeros_like(sh.master)
    sh.from_dense(dense, back)
    real = torch.from_numpy(real_mask(sh)).to(DEV)
    assert torch.equal(back[real], sh.master[real]) and int(back[~real].count_nonzero()) == 0


def test_other_stream_graph_replay_and_repeat_agree():
    sh, twin = make_shard([1000, 37, 50_030], 2, 1, 64), make_shard([1000, 37, 50_030], 2, 1, 64)
    grads = rank_buffers(sh, 4, F16, sh.local_base)
    kw = dict(hyper=HP, rank_grads=grads, grad_base=sh.local_base, divisor=4.0)
    p16, q16 = (torch.zeros(sh.blocks * Q, dtype=torch.float16, device=DEV) for _ in range(2))
    start = make_shard([1000, 37, 50_030], 2, 1, 64)
    sh.adam_step(step=3, param16=p16, param_base=sh.local_base, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        twin.adam_step(step=3, param16=q16, param_base=sh.local_base, **kw)
    torch.cuda.synchronize()
    want = state_bits(sh)
    for x, y in zip(want, state_bits(twin)):
        assert np.array_equal(x, y)
    assert torch.equal(p16.view(torch.int16), q16.view(torch.int16))
    copy_state(start, twin)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        twin.adam_step(step=3, param16=q16, param_base=sh.local_base, **kw)
    for _ in range(3):
        copy_state(start, twin)
        q16.zero_()
        torch.randn(4096, device=DEV).sum()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(want, state_bits(twin)):
            assert np.array_equal(x, y)
        assert torch.equal(p16.view(torch.int16), q16.view(torch.int16))


def test_a_least_squares_fit_follows_the_32_bit_step():
    """300 steps on one least-squares problem: the loss with 8-bit moments ends
    within a factor of two of the loss with 32-bit moments, both far below the start."""
    torch.manual_seed(0)
    n, k = 512, 64
    x = torch.randn(n, k, device=DEV)
    y = x @ torch.randn(k, 32, device=DEV)
    hp = dict(HP, lr=0.05, beta1=0.9, beta2=0.99, weight_decay=0.0)
    end = {}
    for cls in (zs.OwnerShard, zs.OwnerShard8):
        sh = cls([k * 32], 1, 0, align=64, device=DEV)
        sh.alloc_state()
        for step in range(1, 301):
            w = sh.master[:k * 32].view(k, 32)
            e = x @ w - y
            g = (x.t() @ e / n).reshape(-1).contiguous()
            sh.adam_step(step=step, hyper=dict(hp, lr=0.05 * (1 - step / 320)), rank_grads=[g])
        end[cls] = float((x @ sh.master[:k * 32].view(k, 32) - y).square().mean())
    start = float(y.square().mean())
    assert end[zs.OwnerShard] < 1e-3 * start
    assert end[zs.OwnerShard8] < 1e-3 * start


def test_binding_refusals():
    sh = make_shard([1000], 1, 0, 64)
    g = torch.zeros(sh.blocks * Q, device=DEV)
    ok = dict(sh._state8(), master=sh.master, step=1, reduced_g=g, **HP)
    for change, err in ((dict(exp_avg8=sh.exp_avg8.view(torch.uint8)), TypeError),
                        (dict(exp_avg8=sh.exp_avg8[:512]), ValueError),
                        (dict(exp_rms_scale=sh.exp_rms_scale[:1]), ValueError),
                        (dict(master=sh.master[:100]), ValueError), (dict(master=sh.master.half()), TypeError),
                        (dict(reduced_g=g[:10]), ValueError), (dict(reduced_g=g.cpu()), ValueError),
                        (dict(n_pieces=100), ValueError), (dict(param16=g), TypeError),
                        (dict(local_base=8), zs.ZeroShardError), (dict(step=0), zs.ZeroShardError),
                        (dict(beta1=1.0), zs.ZeroShardError)):
        with pytest.raises(err):
            zs.zero_adam8_step(**{**ok, **change})
