"""Token log-probabilities, the clipped policy loss and the preference loss against
their definitions in 64 bits, on the same logits.

Tolerances.  u = 2^-24.  A term exp((x - M) / T) of a row's sum S carries the
rounding of x - M, of the factor log2(e) / T and of their product (together
2.5 u d, d = (M - x) / T), two steps of the exponential and the additions of
one thread's and one wavefront's share, at most K = V / 100 + 80 of them.  So
  ln S is off by at most  e_S = u (2.5 E_p[d] + 4 + K),
  lp by at most           e_S + u |x_t - M| / T (+ half an fp32 step when stored),
  p_j, relative, by       u (2.5 d_j + 6) + e_S,
and what depends on lp follows by its slope.  The store rounds to the logits'
type: eps / 2 relative, or half the smallest subnormal.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import zero_sharded_optimizer_owned_amd as zs  # noqa: E402

DEV = "cuda"
U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SUB = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -126}  # fp32's exponential may flush subnormals
#            rows, vocab, row stride (0: dense), elements before the first row
SHAPES = [(1, 1, 0, 0), (3, 2, 0, 0), (5, 7, 0, 1), (4, 8, 0, 0), (2, 9, 11, 3), (7, 257, 0, 0), (6, 1000, 1024, 0),
          (3, 2047, 0, 5), (5, 4096, 4104, 8), (2, 16_385, 0, 0), (3, 32_000, 0, 0), (2, 50_001, 0, 1),
          (2, 131_072, 0, 0), (1, 131_073, 0, 0), (2, 200_003, 200_004, 2), (1, 400_000, 0, 0)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    zs.lib()
    yield
    torch.cuda.synchronize()


def rows_of(n, v, stride, lead, dtype, seed=0, spread=3.0, special=True):
    """[n, v] logits inside a larger buffer, targets with some rows ignored, masked tokens."""
    g = torch.Generator().manual_seed(seed + 1000 * v + n)
    stride = stride or v
    buf = torch.full((lead + n * stride + 8,), float("nan"))
    x = buf[lead:lead + n * stride].view(n, stride)[:, :v]
    x.copy_(torch.randn(n, v, generator=g) * spread)
    t = torch.randint(0, v, (n,), generator=g)
    x[torch.arange(n), t] += 4.0
    if special and v > 4:
        hide = (t[-1] + 1) % v  # a masked token beside the target, and the type's lowest value
        x[-1, hide] = -math.inf
        x[0, (t[0] + 1) % v] = torch.finfo(dtype).min
    dev = torch.empty(buf.numel() + 64, dtype=dtype, device=DEV)[:buf.numel()]
    dev.copy_(buf.clamp(torch.finfo(dtype).min, None).masked_fill(buf == -math.inf, -math.inf))
    if special and n > 2:
        t[1] = -100
    return dev[lead:lead + n * stride].view(n, stride)[:, :v], t.to(DEV)


def reference(x, t, temperature):
    """float64 on the host: lp, p, its error bounds, which rows count."""
    n, v = x.shape
    x = x.detach().cpu().double()
    t = t.cpu()
    z = x / temperature
    top = z.max(1, keepdim=True).values
    counts = (t >= 0) & (t < v) & (top[:, 0] > -math.inf)
    d = torch.where(torch.isfinite(top), top - z, torch.zeros_like(z))
    e = (-d).exp()
    s = e.sum(1, keepdim=True)
    p = e / s
    at = torch.where(counts, t, torch.zeros_like(t))
    rows = torch.arange(n)
    dt = d[rows, at]
    lp = torch.where(counts, -dt - s[:, 0].log(), torch.zeros_like(dt))
    finite = torch.where(torch.isfinite(d), d, torch.zeros_like(d))
    e_s = U * (2.5 * (p * finite).sum(1) + 4 + v / 100 + 80)
    e_lp = e_s + U * torch.where(torch.isfinite(dt), dt, torch.zeros_like(dt))
    e_p = U * (2.5 * finite + 6) + e_s[:, None]
    return dict(lp=lp, p=p, counts=counts, at=at, e_lp=e_lp, e_p=e_p, n=n, v=v)


def close(got, want, tol, what):
    got = got.detach().cpu().double()
    ok = ((got - want).abs() <= tol) | (got == want)
    assert bool(ok.all()), f"{what}: off at {torch.nonzero(~ok)[:4].tolist()}: {got[~ok][:4]} vs {want[~ok][:4]}"


def check_gradient(ref, dlogits, coef, e_coef, name, what):
    """dlogits against coef ([j = t] - p), coef known to e_coef."""
    hot = torch.zeros(ref["n"], ref["v"], dtype=torch.float64)
    hot[torch.arange(ref["n"]), ref["at"]] = 1.0
    lever = hot - ref["p"]
    want = coef[:, None] * lever
    tol = e_coef[:, None] * lever.abs() + coef.abs()[:, None] * (ref["p"] * ref["e_p"] + 3 * U * hot)
    tol = tol + (want.abs() + tol) * torch.finfo(DT[name]).eps / 2 + SUB[name]
    close(dlogits, want, tol, what)
    assert int(dlogits.detach().cpu()[~ref["counts"]].count_nonzero()) == 0, what


def logp_tol(ref):
    return ref["e_lp"] + U * ref["lp"].abs()


@pytest.mark.parametrize("name", list(DT))
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("temperature", [1.0, 0.6])
def test_logprobs(shape, name, temperature):
    x, t = rows_of(*shape, DT[name])
    out = torch.full((shape[0],), 7.0, device=DEV)
    zs.zero_token_logprobs(x, t, out, temperature=temperature)
    ref = reference(x, t, temperature)
    close(out, ref["lp"], logp_tol(ref), f"{shape} {name}")


def policy_inputs(ref, seed=3):
    g = torch.Generator().manual_seed(seed)
    n = ref["n"]
    d = torch.randn(n, generator=g, dtype=torch.float64) * 0.3
    for border in (math.log(0.8), math.log(1.3)):
        d = torch.where((d - border).abs() < 1e-2, d + 2e-2, d)
    f = lambda x: x.float().to(DEV)
    return dict(old_logp=f(ref["lp"] - d), ref_logp=f(ref["lp"] + 0.2 * torch.randn(n, generator=g, dtype=torch.float64)),
                advantage=f(torch.randn(n, generator=g)), weight=f(torch.rand(n, generator=g) + 0.1))


def policy_reference(ref, inp, divisor, low, high, kl, temperature, scale):
    h = {k: v.cpu().double() for k, v in inp.items() if v is not None}
    w = h.get("weight", torch.ones(ref["n"], dtype=torch.float64)) * ref["counts"] / divisor
    a, lp = h["advantage"], ref["lp"]
    ratio = (lp - h["old_logp"]).exp()
    free, held = a * ratio, a * ratio.clamp(1 - low, 1 + high)
    clipped = held < free
    gain = torch.minimum(free, held)
    d = h["ref_logp"] - lp if "ref_logp" in h else torch.zeros_like(lp)
    k3 = torch.expm1(d) - d
    live = w != 0
    z = lambda x: torch.where(live, x, torch.zeros_like(x))
    pg, k3s, cl = z(-w * gain).sum(), z(w * k3).sum(), z(w * clipped).sum()
    slope = torch.where(clipped, torch.zeros_like(free), -free) - kl * torch.expm1(d)
    gain_slope = free.abs() * ~clipped + kl * d.exp()
    f = scale / temperature
    coef, e_coef = z(w * slope * f), z(w * (gain_slope * ref["e_lp"] * 1.01 + slope.abs() * 2 * U) * f)
    stats = torch.stack([pg + kl * k3s, pg, k3s, cl])
    e_pg = z(w * free.abs() * ~clipped * ref["e_lp"]).sum() * 1.01
    e_kl = z(w * torch.expm1(d).abs() * ref["e_lp"]).sum() * 1.01 + z(w * ref["e_lp"] ** 2).sum()
    e_stats = torch.stack([e_pg + kl * e_kl, e_pg, e_kl, torch.zeros(())]) + 2 * U * stats.abs()
    return stats, e_stats, coef, e_coef


@pytest.mark.parametrize("name", list(DT))
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kl, temperature, plain", [(0.05, 1.0, False), (0.0, 0.6, True)])
def test_policy_loss_and_gradient(shape, name, kl, temperature, plain):
    x, t = rows_of(*shape, DT[name])
    ref = reference(x, t, temperature)
    inp = policy_inputs(ref)
    if plain:  # no reference model, every row of weight 1
        inp["ref_logp"] = inp["weight"] = None
    n, v = x.shape
    stats, logp = torch.full((4,), 9.0, device=DEV), torch.full((n,), 9.0, device=DEV)
    whole = torch.full_like(x.as_strided((n, x.stride(0)), (x.stride(0), 1)) if x.stride(0) > v and n > 1 else x, 5.0)
    dx = whole[:, :v]
    scale = 64.0 if name == "f16" else 1.0
    zs.zero_policy_loss(x, t, divisor=3.0, stats=stats, logp=logp, workspace=zs.policy_workspace(n, DEV), clip_low=0.2,
                        clip_high=0.3, kl_coef=kl, temperature=temperature, grad_scale=scale, dlogits=dx, **inp)
    want, e_want, coef, e_coef = policy_reference(ref, inp, 3.0, 0.2, 0.3, kl, temperature, scale)
    close(logp, ref["lp"], logp_tol(ref), "logp")
    close(stats, want, e_want, "stats")
    check_gradient(ref, dx, coef, e_coef, name, f"{shape} {name}")
    assert bool((whole[:, v:] == 5.0).all()), "wrote between the rows"


def packed(lengths, v, name, seed=0):
    n = sum(lengths)
    x, t = rows_of(n, v, 0, 0, DT[name], seed=seed, special=False)
    skip = torch.rand(n, generator=torch.Generator().manual_seed(seed)) < 0.2
    t[skip.to(DEV)] = -100
    return x, t, torch.tensor([0] + lengths).cumsum(0).to(DEV)


def preference_reference(ref, bounds, ref_logp, beta, eps, average, temperature, scale):
    b = bounds.cpu().tolist()
    pairs = len(b) // 2
    e_row = torch.where(ref["counts"], ref["e_lp"], torch.zeros_like(ref["e_lp"]))
    s, e, part = [], [], []
    for q in range(2 * pairs):
        rows = slice(b[q], b[q + 1])
        k = max(1, int(ref["counts"][rows].sum())) if average else 1
        s.append(ref["lp"][rows].sum() / k)
        e.append(e_row[rows].sum() / k)
        part.append(1.0 / k)
    s, e, part = torch.stack(s), torch.stack(e), torch.tensor(part, dtype=torch.float64)
    reward = beta * (s - ref_logp.cpu().double() * part)
    h, e_h = reward[0::2] - reward[1::2], beta * (e[0::2] + e[1::2]) + 1e-12
    ls = torch.nn.functional.logsigmoid
    loss = -((1 - eps) * ls(h) + eps * ls(-h))
    slope = beta / pairs * (torch.sigmoid(h) - (1 - eps)) * scale / temperature
    e_slope = beta / pairs * 0.25 * e_h * scale / temperature + 2 * U * slope.abs()
    coef, e_coef = (torch.zeros(ref["n"], dtype=torch.float64) for _ in range(2))
    for q in range(2 * pairs):
        rows = slice(b[q], b[q + 1])
        coef[rows] = slope[q // 2] * part[q] * (1 - 2 * (q % 2))
        e_coef[rows] = e_slope[q // 2] * part[q]
    coef, e_coef = coef * ref["counts"], e_coef * ref["counts"]
    return dict(seq=s, e_seq=e + U * s.abs(), reward=reward, e_reward=beta * e + U * reward.abs() + 1e-12,
                stats=torch.stack([loss.mean(), (h > 0).double().mean()]),
                e_stats=torch.stack([e_h.mean() + U * loss.mean(), torch.zeros((), dtype=torch.float64)]),
                coef=coef, e_coef=e_coef, h=h, e_h=e_h)


@pytest.mark.parametrize("name", list(DT))
@pytest.mark.parametrize("lengths, v", [([1, 1], 5), ([3, 2, 1, 6], 100), ([0, 4, 3, 0], 33), ([300, 17], 257),
                                        ([40, 41, 5, 90, 7, 7], 5000), ([2, 3], 140_001)])
@pytest.mark.parametrize("average, eps, temperature", [(False, 0.0, 1.0), (True, 0.1, 0.8)])
def test_preference_loss_and_gradient(lengths, v, name, average, eps, temperature):
    x, t, bounds = packed(lengths, v, name)
    ref = reference(x, t, temperature)
    n, q = len(t), len(lengths)
    g = torch.Generator().manual_seed(8)
    sums = torch.stack([ref["lp"][a:b].sum() for a, b in zip(bounds.tolist(), bounds.tolist()[1:])])
    ref_logp = (sums + 2 * torch.randn(q, generator=g, dtype=torch.float64)).float().to(DEV)
    mk = lambda k: torch.full((k,), 9.0, device=DEV)
    stats, logp, seq, reward, dx = mk(2), mk(n), mk(q), mk(q), torch.full_like(x, 5.0)
    scale = 256.0 if name == "f16" else 1.0
    zs.zero_preference_loss(x, t, bounds, ref_logp=ref_logp, stats=stats, logp=logp, seq_logp=seq, reward=reward,
                            workspace=zs.preference_workspace(n, q // 2, DEV), beta=0.3, label_smoothing=eps,
                            average=average, temperature=temperature, grad_scale=scale, dlogits=dx)
    want = preference_reference(ref, bounds, ref_logp, 0.3, eps, average, temperature, scale)
    close(logp, ref["lp"], logp_tol(ref), "logp")
    close(seq, want["seq"], want["e_seq"], "seq_logp")
    close(reward, want["reward"], want["e_reward"], "reward")
    assert bool((want["h"].abs() > want["e_h"]).all())  # the pairs' order is not a matter of rounding
    close(stats, want["stats"], want["e_stats"], "stats")
    check_gradient(ref, dx, want["coef"], want["e_coef"], name, str(lengths))


def run_policy(x, t, dx=None, kl=0.1, seed=3, **over):
    n = x.shape[0]
    ref = reference(x, t, 1.0)
    inp = {**policy_inputs(ref, seed), **over}
    stats, logp = torch.zeros(4, device=DEV), torch.zeros(n, device=DEV)
    zs.zero_policy_loss(x, t, divisor=1.0, stats=stats, logp=logp, workspace=zs.policy_workspace(n, DEV), clip_low=0.2,
                        clip_high=0.3, kl_coef=kl, dlogits=dx, **inp)
    return stats, logp


@pytest.mark.parametrize("name", list(DT))
@pytest.mark.parametrize("v", [513, 32_000, 131_072, 131_081])
def test_gradient_in_place_and_at_another_alignment(name, v):
    """dlogits may be the logits themselves, or rows of another 16-byte phase: the same bits."""
    x, t = rows_of(4, v, 0, 0, DT[name])
    dx = torch.empty_like(x)
    want = run_policy(x, t, dx)
    off = torch.empty(4 * (v + 3) + 5, dtype=DT[name], device=DEV)[1:1 + 4 * (v + 3)].view(4, v + 3)[:, :v]
    inplace = x.clone()
    for out, src in ((off, x), (inplace, inplace)):
        got = run_policy(src, t, out) if src is x else None
        if got is None:
            ref_in = policy_inputs(reference(x, t, 1.0))
            got = torch.zeros(4, device=DEV), torch.zeros(4, device=DEV)
            zs.zero_policy_loss(inplace, t, divisor=1.0, stats=got[0], logp=got[1],
                                workspace=zs.policy_workspace(4, DEV), clip_low=0.2, clip_high=0.3, kl_coef=0.1,
                                dlogits=inplace, **ref_in)
        bits = lambda y: y.contiguous().view(torch.uint8)
        assert torch.equal(bits(out), bits(dx))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_gradient_of_preference_in_place():
    x, t, bounds = packed([40, 41, 5, 90], 5000, "bf16")
    n = len(t)
    outs = []
    for inplace in (False, True):
        y = x.clone()
        dx = y if inplace else torch.empty_like(y)
        mk = lambda k: torch.zeros(k, device=DEV)
        zs.zero_preference_loss(y, t, bounds, ref_logp=mk(4), stats=mk(2), logp=mk(n), seq_logp=mk(4), reward=mk(4),
                                workspace=zs.preference_workspace(n, 2, DEV), dlogits=dx)
        outs.append(dx.view(torch.int16).clone())
    assert torch.equal(*outs)


@pytest.mark.parametrize("v", [9, 40_000, 140_000])
def test_rows_that_leave_nothing(v):
    """All -inf, an ignored row full of NaN, and a row with NaN at weight 0: no loss, zero gradient."""
    x, t = rows_of(6, v, 0, 0, torch.float32, special=False)
    x[1] = -math.inf
    x[2] = math.nan
    t[2] = -100
    x[3] = torch.finfo(torch.float32).min  # all the lowest value: a uniform row
    t[4] = v  # outside the vocabulary
    ref_in = policy_inputs(reference(x[:, :], t, 1.0))
    ref_in["advantage"][1] = ref_in["advantage"][2] = ref_in["old_logp"][4] = math.nan  # not looked at
    dx, stats, logp = torch.full_like(x, 5.0), torch.zeros(4, device=DEV), torch.full((6,), 5.0, device=DEV)
    zs.zero_policy_loss(x, t, divisor=1.0, stats=stats, logp=logp, workspace=zs.policy_workspace(6, DEV), kl_coef=0.1,
                        dlogits=dx, **ref_in)
    assert bool(torch.isfinite(stats).all())
    for row in (1, 2, 4):
        assert float(logp[row]) == 0.0 and int(dx[row].count_nonzero()) == 0
    assert abs(float(logp[3]) + math.log(v)) <= 1e-5
    assert bool(torch.isfinite(dx).all())
    out = torch.full((6,), 5.0, device=DEV)
    zs.zero_token_logprobs(x, t, out)
    assert torch.equal(out, logp)
    ref_in["weight"][5] = 0.0
    ref_in["advantage"][5] = math.nan
    zs.zero_policy_loss(x, t, divisor=1.0, stats=stats, logp=logp, workspace=zs.policy_workspace(6, DEV), kl_coef=0.1,
                        dlogits=dx, **ref_in)
    assert bool(torch.isfinite(stats).all()) and int(dx[5].count_nonzero()) == 0


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("v", [9, 40_000, 140_000])
def test_non_finite_logits_show_in_their_row_alone(bad, v):
    x, t = rows_of(4, v, 0, 0, torch.float32, special=False)
    x[2, (t[2] + 3) % v] = bad
    dx = torch.zeros_like(x)
    ref_in = policy_inputs(dict(reference(torch.nan_to_num(x, 0, 0), t, 1.0)))
    stats, logp = torch.zeros(4, device=DEV), torch.zeros(4, device=DEV)
    zs.zero_policy_loss(x, t, divisor=1.0, stats=stats, logp=logp, workspace=zs.policy_workspace(4, DEV), kl_coef=0.1,
                        dlogits=dx, **ref_in)
    assert math.isnan(float(stats[0])) and math.isnan(float(logp[2]))
    fine = [0, 1, 3]
    assert bool(torch.isfinite(dx[fine]).all()) and not bool(torch.isfinite(dx[2]).any())


def test_a_target_of_minus_infinity():
    """Its log-probability is -inf; the ratio is 0, and the row's gradient is finite without a KL term."""
    x, t = rows_of(3, 100, 0, 0, torch.bfloat16, special=False)
    x[1, t[1]] = -math.inf
    out = torch.zeros(3, device=DEV)
    zs.zero_token_logprobs(x, t, out)
    assert float(out[1]) == -math.inf and bool(torch.isfinite(out[[0, 2]]).all())
    f = lambda *v: torch.tensor(v, device=DEV)
    dx, stats = torch.zeros_like(x), torch.zeros(4, device=DEV)
    zs.zero_policy_loss(x, t, old_logp=f(-1.0, -1.0, -1.0), advantage=f(1.0, 2.0, -1.0), divisor=1.0, stats=stats,
                        logp=out, workspace=zs.policy_workspace(3, DEV), dlogits=dx)
    assert bool(torch.isfinite(stats).all()) and bool(torch.isfinite(dx).all()) and int(dx[1].count_nonzero()) == 0


def test_overflowing_ratios():
    """A zero advantage takes nothing of an infinite ratio; a positive one is clipped."""
    x, t = rows_of(2, 50, 0, 0, torch.float32, special=False)
    f = lambda *v: torch.tensor(v, device=DEV)
    dx, stats, logp = torch.ones_like(x), torch.zeros(4, device=DEV), torch.zeros(2, device=DEV)
    zs.zero_policy_loss(x, t, old_logp=f(-1e4, -1e4), advantage=f(0.0, 2.0), divisor=1.0, stats=stats, logp=logp,
                        workspace=zs.policy_workspace(2, DEV), dlogits=dx)
    assert abs(float(stats[0]) + 2.4) < 1e-6 and float(stats[3]) == 1.0
    assert int(dx.count_nonzero()) == 0


def test_no_rows():
    x, t = torch.zeros(0, 10, device=DEV), torch.zeros(0, dtype=torch.int64, device=DEV)
    e, stats = torch.zeros(0, device=DEV), torch.full((4,), 9.0, device=DEV)
    zs.zero_token_logprobs(x, t, e)
    zs.zero_policy_loss(x, t, old_logp=e, advantage=e, divisor=1.0, stats=stats, logp=e, dlogits=torch.zeros_like(x),
                        workspace=zs.policy_workspace(0, DEV))
    assert stats.tolist() == [0.0] * 4
    s2 = torch.full((2,), 9.0, device=DEV)
    seq, reward = s2.clone(), s2.clone()
    zs.zero_preference_loss(x, t, torch.zeros(3, dtype=torch.int64, device=DEV), ref_logp=torch.zeros(2, device=DEV),
                            stats=s2, logp=e, seq_logp=seq, reward=reward, dlogits=torch.zeros_like(x),
                            workspace=zs.preference_workspace(0, 1, DEV))
    assert abs(float(s2[0]) - math.log(2)) < 1e-6 and seq.tolist() == [0.0, 0.0]


def test_rows_outside_every_sequence_and_boundaries_outside_the_rows():
    x, t, _ = packed([10, 10], 64, "f32", seed=2)
    bounds = torch.tensor([4, 9, 1000], device=DEV)
    mk = lambda k: torch.zeros(k, device=DEV)
    dx, logp = torch.full_like(x, 5.0), mk(20)
    zs.zero_preference_loss(x, t, bounds, ref_logp=mk(2), stats=mk(2), logp=logp, seq_logp=mk(2), reward=mk(2),
                            workspace=zs.preference_workspace(20, 1, DEV), dlogits=dx)
    ref = reference(x, t, 1.0)
    close(logp, ref["lp"], logp_tol(ref), "logp")
    want = preference_reference(ref, torch.tensor([4, 9, 20]), torch.zeros(2), 0.1, 0.0, False, 1.0, 1.0)
    check_gradient(ref, dx, want["coef"], want["e_coef"], "f32", "outside")
    assert int(dx[:4].count_nonzero()) == 0


def test_gradients_against_differences():
    """Central differences of the kernels' own losses along a random direction.  With
    steps of 1e-2 the loss's fp32 rounding is 2^-24 |loss| / 1e-2 and the third-order
    term about 1e-4 of the slope."""
    g = torch.Generator().manual_seed(5)
    x, t = rows_of(6, 37, 0, 0, torch.float32, special=False, spread=1.0)
    u = torch.randn(6, 37, generator=g).to(DEV)
    u /= u.norm()
    inp = policy_inputs(reference(x, t, 1.0))
    inp["old_logp"] = (reference(x, t, 1.0)["lp"] - 0.1 * torch.tensor([1, -1, 0.5, -0.5, 0, 1])).float().to(DEV)
    ws = zs.policy_workspace(6, DEV)

    def policy_value(y, dx=None):
        stats = torch.zeros(4, device=DEV)
        zs.zero_policy_loss(y, t, divisor=2.0, stats=stats, logp=torch.zeros(6, device=DEV), workspace=ws, kl_coef=0.3,
                            dlogits=dx, **inp)
        return float(stats[0])

    bounds, ref_logp = torch.tensor([0, 2, 3, 4, 6], device=DEV), torch.tensor([-4.0, -5.0, -3.0, -6.0], device=DEV)
    ws2 = zs.preference_workspace(6, 2, DEV)

    def preference_value(y, dx=None):
        mk = lambda k: torch.zeros(k, device=DEV)
        stats = mk(2)
        zs.zero_preference_loss(y, t, bounds, ref_logp=ref_logp, stats=stats, logp=mk(6), seq_logp=mk(4), reward=mk(4),
                                workspace=ws2, beta=0.7, label_smoothing=0.1, dlogits=dx)
        return float(stats[0])

    for value in (policy_value, preference_value):
        dx = torch.zeros_like(x)
        loss = value(x, dx)
        slope = float((dx.double() * u.double()).sum())
        got = (value(x + 1e-2 * u) - value(x - 1e-2 * u)) / 2e-2
        assert abs(got - slope) <= 2 * 2 ** -24 * abs(loss) / 1e-2 + 1e-3 * float(dx.norm())


def test_offsets_beyond_32_bits():
    """Rows more than 2^32 elements apart."""
    v, stride = 1000, 2_200_000_000
    buf = torch.empty(2 * stride + v, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((3, v), (stride, 1))
    x.copy_(torch.randn(3, v, generator=torch.Generator().manual_seed(1)))
    t = torch.tensor([5, 999, 0], device=DEV)
    out = torch.zeros(3, device=DEV)
    zs.zero_token_logprobs(x, t, out)
    ref = reference(x, t, 1.0)
    close(out, ref["lp"], logp_tol(ref), "logp")
    stats, logp = run_policy(x, t, dx=x)
    close(logp, ref["lp"], logp_tol(ref), "logp")
    del buf, x
    torch.cuda.empty_cache()


def test_many_rows_repeat_and_run_on_another_stream_alike():
    x, t = rows_of(5000, 129, 0, 0, torch.bfloat16)
    dx, dy = torch.empty_like(x), torch.empty_like(x)
    want = run_policy(x, t, dx)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run_policy(x, t, dy)
    torch.cuda.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert torch.equal(dx.view(torch.int16), dy.view(torch.int16))


@pytest.mark.parametrize("v", [999, 131_072, 150_000])
def test_graph_replays_like_eager(v):
    x, t = rows_of(64, v, 0, 0, torch.bfloat16)
    keep = x.clone()
    inp = policy_inputs(reference(x, t, 1.0))
    bounds = torch.tensor([0, 10, 30, 31, 64], device=DEV)
    mk = lambda k: torch.zeros(k, device=DEV)
    outs = [mk(4), mk(64), torch.zeros_like(x), mk(2), mk(64), mk(4), mk(4), torch.zeros_like(x)]
    ws, ws2 = zs.policy_workspace(64, DEV), zs.preference_workspace(64, 2, DEV)
    ref_logp = torch.full((4,), -50.0, device=DEV)

    def both():
        zs.zero_policy_loss(x, t, divisor=1.0, stats=outs[0], logp=outs[1], dlogits=outs[2], workspace=ws, kl_coef=0.1,
                            **inp)
        zs.zero_preference_loss(x, t, bounds, ref_logp=ref_logp, stats=outs[3], logp=outs[4], seq_logp=outs[5],
                                reward=outs[6], dlogits=outs[7], workspace=ws2)

    both()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for _ in range(3):
        for o in outs:
            o.fill_(3.0)
        x.copy_(keep)
        torch.randn(4096, device=DEV).sum()
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


def test_binding_refusals():
    x, t = torch.zeros(3, 8, device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV)
    o = torch.zeros(4, device=DEV)
    ws = zs.policy_workspace(3, DEV)
    ok = dict(old_logp=o, advantage=o, divisor=1.0, stats=o.clone(), logp=o.clone(), workspace=ws)
    with pytest.raises(ValueError):
        zs.zero_token_logprobs(x.t(), torch.zeros(8, dtype=torch.int64, device=DEV), torch.zeros(8, device=DEV))
    with pytest.raises(TypeError):
        zs.zero_token_logprobs(x, t.int(), o)
    with pytest.raises(ValueError):
        zs.zero_token_logprobs(x, t[:2], o)
    with pytest.raises(ValueError):
        zs.zero_token_logprobs(x, t, o[:2])
    for change, err in ((dict(old_logp=o[:2]), ValueError), (dict(advantage=o.double()), TypeError),
                        (dict(stats=o[:3]), ValueError), (dict(dlogits=x.half()), ValueError),
                        (dict(dlogits=x[:2]), ValueError), (dict(kl_coef=0.1), zs.ZeroShardError),
                        (dict(workspace=ws[:8].clone()), zs.ZeroShardError), (dict(divisor=0.0), zs.ZeroShardError)):
        with pytest.raises(err):
            zs.zero_policy_loss(x, t, **{**ok, **change})
    with pytest.raises(ValueError):
        zs.zero_token_logprobs(x[:1].expand(3, 8), t, o)  # overlapping rows


def test_more_rows_than_one_launch_takes():
    """2^21 rows and a few: the rows of the second launch equal a call on them alone."""
    n, v, cut = (1 << 21) + 5, 128, 1 << 21
    g = torch.Generator(DEV).manual_seed(3)
    x = torch.randn(n, v, generator=g, device=DEV).half()
    t = torch.randint(0, v, (n,), generator=g, device=DEV)
    a, b, c = torch.empty(n, device=DEV), torch.empty(n, device=DEV), torch.empty(5, device=DEV)
    zs.zero_token_logprobs(x, t, a)
    zs.zero_token_logprobs(x[cut:], t[cut:], c)
    assert torch.equal(a[cut:], c)
    adv, old = torch.randn(n, generator=g, device=DEV), a - 0.1
    dx, few = torch.empty_like(x), torch.empty_like(x[cut:])
    stats, s2 = torch.zeros(4, device=DEV), torch.zeros(4, device=DEV)
    zs.zero_policy_loss(x, t, old_logp=old, advantage=adv, divisor=1.0, stats=stats, logp=b, dlogits=dx,
                        workspace=zs.policy_workspace(n, DEV))
    assert torch.equal(a, b)
    zs.zero_policy_loss(x[cut:], t[cut:], old_logp=old[cut:], advantage=adv[cut:], divisor=1.0, stats=s2, logp=c,
                        dlogits=few, workspace=zs.policy_workspace(5, DEV))
    assert torch.equal(dx[cut:].view(torch.int16), few.view(torch.int16))
    ratio = (a - old).double().exp()
    gain = torch.minimum(adv * ratio, adv * ratio.clamp(0.8, 1.2)).sum()
    assert abs(float(stats[0]) + float(gain)) <= 1e-6 * float((adv * ratio).abs().sum())


def test_workspace_serves_calls_of_any_smaller_size():
    """One workspace for calls of different row counts, one after the other."""
    ws = zs.policy_workspace(3000, DEV)
    for n in (3000, 7, 128, 129, 1, 3000):
        x, t = rows_of(n, 200, 0, 0, torch.float32)
        inp = policy_inputs(reference(x, t, 1.0))
        got, want = torch.zeros(4, device=DEV), torch.zeros(4, device=DEV)
        for stats, w in ((got, ws), (want, zs.policy_workspace(n, DEV))):
            zs.zero_policy_loss(x, t, divisor=1.0, stats=stats, logp=torch.zeros(n, device=DEV), workspace=w,
                                kl_coef=0.1, **inp)
        assert torch.equal(got, want) and float(want[2]) > 0


def test_many_pairs_take_the_pair_launch_and_agree_with_few():
    """The launch for the pairs (more than 16 pairs or 1024 rows) and the form without it: the same
    rows give the same gradient up to the number of pairs that the loss is divided by."""
    lengths = [5, 3] * 40
    x, t, bounds = packed(lengths, 300, "f32", seed=4)
    n, q = len(t), len(lengths)
    mk = lambda k: torch.zeros(k, device=DEV)
    ref_logp = -torch.arange(q, device=DEV, dtype=torch.float32) * 0.1 - 20
    dx, seq, reward = torch.empty_like(x), mk(q), mk(q)
    zs.zero_preference_loss(x, t, bounds, ref_logp=ref_logp, stats=mk(2), logp=mk(n), seq_logp=seq, reward=reward,
                            workspace=zs.preference_workspace(n, q // 2, DEV), dlogits=dx)
    ref = reference(x, t, 1.0)
    want = preference_reference(ref, bounds, ref_logp, 0.1, 0.0, False, 1.0, 1.0)
    check_gradient(ref, dx, want["coef"], want["e_coef"], "f32", "many pairs")
    k = int(bounds[20])
    few, s2, r2 = torch.empty_like(x[:k]), mk(20), mk(20)
    zs.zero_preference_loss(x[:k], t[:k], bounds[:21], ref_logp=ref_logp[:20], stats=mk(2), logp=mk(k), seq_logp=s2,
                            reward=r2, workspace=zs.preference_workspace(k, 10, DEV), dlogits=few)
    assert torch.equal(s2, seq[:20]) and torch.equal(r2, reward[:20])
    # 40 pairs against 10: a factor of 4, a power of two; the coefficient rounds once in both
    assert torch.equal(few, dx[:k] * 4)
