"""The losses where their rows leave the ordinary: logits far from zero, targets at the
types' ends, low and high temperatures, long rows.

Tolerances.  u = 2^-24.  With the target's logit as the reference, a term
exp((x_j - x_t) / T), d_j = |x_j - x_t| / T, carries the rounding of the difference and of
the exponent (2 u d_j) and one step of the exponential (2 u).  A thread adds a vector's 8
elements and the partial sums of at most 16 vectors in fp32 (24 u), everything past those
in fp64.  So ln S is off by at most u (2 E_p[d] + 26); lp = -ln S is stored in fp32.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import zero_sharded_optimizer_owned_amd as zs  # noqa: E402

DEV = "cuda"
U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    zs.lib()
    yield
    torch.cuda.synchronize()


def full(*shape, value=9.0):
    return torch.full(shape, value, device=DEV)


def logprobs(x, t, temperature=1.0):
    out = full(len(t))
    zs.zero_token_logprobs(x, t, out, temperature=temperature)
    return out


def policy(x, t, old, advantage, temperature=1.0, ref=None, kl=0.0, gradient=True):
    """(stats, logp, dlogits) of the policy loss."""
    stats, logp, dx = full(4), full(len(t)), torch.full_like(x, 5.0) if gradient else None
    zs.zero_policy_loss(x, t, old_logp=old, ref_logp=ref, kl_coef=kl, advantage=advantage, divisor=1.0, stats=stats,
                        logp=logp, dlogits=dx, temperature=temperature, workspace=zs.policy_workspace(len(t), DEV))
    return stats, logp, dx


def preference(x, t, bounds, ref, gradient=True, **over):
    """(stats, logp, seq_logp, reward, dlogits) of the preference loss."""
    q = len(bounds) - 1
    out = full(2), full(len(t)), full(q), full(q), torch.full_like(x, 5.0) if gradient else None
    zs.zero_preference_loss(x, t, bounds, ref_logp=ref, stats=out[0], logp=out[1], seq_logp=out[2], reward=out[3],
                            dlogits=out[4], workspace=zs.preference_workspace(len(t), q // 2, DEV), **over)
    return out


def bits(x):
    return x.contiguous().view(torch.uint8)


def exact_logp(x, t, temperature=1.0):
    """(lp in 64 bits, its tolerance) of every row, by the definition."""
    at = torch.arange(len(t), device=x.device), t
    z = (x.double() - x.double()[at][:, None]) / temperature
    top = z.max(1, keepdim=True).values
    e = (z - top).exp()
    total = e.sum(1)
    lp = -top[:, 0] - total.log()
    spread = (e * torch.where(e > 0, z.abs(), 0.0)).sum(1) / total
    return lp, U * (2 * spread + 26) + U * lp.abs()


def grid_rows(n, v, step, seed=1):
    """Logits at multiples of `step` within +-15 (so that a shift leaves them exact), and targets."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(n, v, generator=g) * 3 / step).round().clamp(-15 / step, 15 / step) * step
    t = torch.randint(0, v, (n,), generator=g)
    x[torch.arange(n), t] = (x[torch.arange(n), t] + 8).clamp(max=15)
    return x.to(DEV), t.to(DEV)


@pytest.mark.parametrize("v", [100, 1000, 8001, 32_000, 131_072, 140_003])
@pytest.mark.parametrize("name, shift, step", [("f32", 1000.0, 2.0 ** -6), ("f32", -4096.0, 2.0 ** -6),
                                               ("f16", 100.0, 2.0 ** -4), ("bf16", 96.0, 0.5), ("bf16", -96.0, 0.5)])
def test_a_common_shift_of_the_logits_changes_nothing(name, shift, step, v):
    """All results are functions of the differences, which are exact here: the same bits."""
    x, t = grid_rows(5, v, step)
    near, far = x.to(DT[name]), (x + shift).to(DT[name])
    assert torch.equal(near.double() + shift, far.double())
    want, tol = exact_logp(near, t)
    adv = torch.tensor([1.0, -0.5, 2.0, 0.25, -1.0], device=DEV)
    old = (want - 0.1).float()
    bounds = torch.tensor([0, 2, 5], device=DEV)
    ref = full(2, value=-20.0)
    a = [logprobs(near, t), *policy(near, t, old, adv, ref=old, kl=0.1), *preference(near, t, bounds, ref)]
    b = [logprobs(far, t), *policy(far, t, old, adv, ref=old, kl=0.1), *preference(far, t, bounds, ref)]
    assert bool(((b[0].double() - want).abs() <= tol).all()), (b[0].double() - want, tol)
    for p, q in zip(a, b):
        assert torch.equal(bits(p), bits(q))


@pytest.mark.parametrize("v", [64, 1000, 50_001, 140_000])
@pytest.mark.parametrize("name", list(DT))
def test_the_calls_agree_on_a_token(name, v):
    """The reference's sums and the policy's: one log-probability, whichever call forms it."""
    x, t = grid_rows(6, v, 0.5, seed=2)
    x = (x + 17).to(DT[name])
    x[4, (t[4] + 1) % v] = 100.0  # a row whose maximum is far above its target
    lp = logprobs(x, t)
    want, tol = exact_logp(x, t)
    assert bool(((lp.double() - want).abs() <= tol).all())
    stats, again, dx = policy(x, t, lp, full(6, value=1.0), ref=lp, kl=0.5)
    assert torch.equal(lp, again)
    _, third, _, _, _ = preference(x, t, torch.tensor([0, 3, 6], device=DEV), full(2, value=0.0))
    assert torch.equal(lp, third)


@pytest.mark.parametrize("temperature", [0.1, 0.02])
@pytest.mark.parametrize("v", [90, 4096, 131_072])
def test_low_temperatures(v, temperature):
    """Near-certain targets: no log-probability above zero, all within the bound."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn(8, v, generator=g) * 2
    t = torch.randint(0, v, (8,), generator=g)
    t[6:] = t[6:].clamp(min=1)
    x[torch.arange(8), t] = 30.0 + torch.rand(8, generator=g)
    x[6:, 0] = 12.0  # one row's target below its maximum, one far below
    x[6, t[6]], x[7, t[7]] = 10.5, -3.0
    x, t = x.to(DEV), t.to(DEV)
    want, tol = exact_logp(x, t, temperature)
    got = logprobs(x, t, temperature)
    assert bool((got <= 0).all()), got
    assert bool(((got.double() - want).abs() <= tol).all()), (got.double() - want, tol)
    assert torch.equal(policy(x, t, got, full(8, value=1.0), temperature)[1], got)


@pytest.mark.parametrize("v", [9, 1000, 40_000, 131_072, 140_000])
@pytest.mark.parametrize("name", ["bf16", "f32"])
@pytest.mark.parametrize("temperature", [1.0, 0.6])
def test_a_target_at_the_types_largest_value(name, v, temperature):
    """It is certain: lp 0, and with it the gradient; beside a second one it has half."""
    x, t = grid_rows(4, v, 0.5, seed=3)
    x = x.to(DT[name])
    big = torch.finfo(DT[name]).max
    for row in (0, 1, 3):
        x[row, t[row]] = big
    x[1, (t[1] + 1) % v] = big
    x[3] = torch.finfo(DT[name]).min
    x[3, t[3]] = big  # differences beyond fp32
    lp = logprobs(x, t, temperature)
    assert float(lp[0]) == 0.0 and float(lp[3]) == 0.0
    assert abs(float(lp[1]) + math.log(2)) <= 2 * U
    old = full(4, value=0.0)
    old[2] = lp[2]
    stats, again, dx = policy(x, t, old, full(4, value=1.0), temperature)
    assert torch.equal(lp, again) and bool(torch.isfinite(dx).all()) and bool(torch.isfinite(stats).all())
    assert int(dx[[0, 3]].count_nonzero()) == 0 and int(dx[1].count_nonzero()) == 2
    assert abs(float(stats[1]) + 3.5) <= 4 * U * 3.5 + 1e-6  # rows 0, 2, 3 at ratio 1, row 1 at 1/2
    lp3 = preference(x, t, torch.tensor([0, 2, 4], device=DEV), full(2, value=0.0), temperature=temperature)[1]
    assert torch.equal(lp, lp3)


def test_a_target_at_the_lowest_value_beside_the_largest():
    """The difference is beyond fp32, its quotient by the temperature is not."""
    x, t = torch.zeros(2, 300, device=DEV), torch.tensor([4, 7], device=DEV)
    x[0, 4], x[0, 5] = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
    got = logprobs(x, t, temperature=4.0)
    want = 2.0 * torch.finfo(torch.float32).min / 4.0
    assert abs(float(got[0]) - want) <= abs(want) * 2 * U


@pytest.mark.parametrize("temperature", [1e6, 3.7e37, 4.4e37, 6e37, 1e38])
@pytest.mark.parametrize("v", [50, 3000])
def test_high_temperatures_and_masked_tokens(v, temperature):
    """Every unmasked token is as likely as any other; masked ones are not counted."""
    x, t = grid_rows(3, v, 0.5, seed=5)
    x[1, (t[1] + 1) % v] = -math.inf
    t[2] = 0
    x[2, 1:] = -math.inf
    lp = logprobs(x, t, temperature)
    for row, n in enumerate((v, v - 1, 1)):
        assert abs(float(lp[row]) + math.log(n)) <= U * (26 + math.log(n)) + 30 / temperature
    assert torch.equal(lp, policy(x, t, lp, full(3, value=1.0), temperature)[1])


@pytest.mark.parametrize("pairs", [2, 40])  # with the pairs in the gradient's launch, and in one of their own
@pytest.mark.parametrize("smoothing", [0.0, 0.1])
def test_a_masked_target_in_a_pair(pairs, smoothing):
    """A rejected answer of probability 0 leaves no loss and no gradient (with smoothing, an infinite loss: its
    -ln sigma(-h) counts); a chosen one an infinite loss and the full slope."""
    v, n = 200, 4 * pairs  # two tokens to a sequence
    x, t = grid_rows(n, v, 0.5, seed=6)
    bounds, ref = torch.arange(0, n + 1, 2, device=DEV), full(2 * pairs, value=-9.0)
    plain = preference(x, t, bounds, ref, label_smoothing=smoothing)
    y = x.clone()
    y[3, t[3]] = -math.inf  # pair 0's rejected sequence
    stats, logp, seq, reward, dx = preference(y, t, bounds, ref, label_smoothing=smoothing)
    assert float(logp[3]) == float(seq[1]) == float(reward[1]) == -math.inf
    others = [q for q in range(2 * pairs) if q != 1]
    assert torch.equal(reward[others], plain[3][others])
    h = (reward[0::2] - reward[1::2]).double()[1:]
    rest = -((1 - smoothing) * torch.nn.functional.logsigmoid(h) + smoothing * torch.nn.functional.logsigmoid(-h)).sum()
    if smoothing == 0.0:
        assert abs(float(stats[0]) - float(rest) / pairs) <= 1e-6
        assert int(dx[:4].count_nonzero()) == 0
    else:
        assert float(stats[0]) == math.inf and bool(torch.isfinite(dx).all())
        assert torch.equal(dx[4:], plain[4][4:])
    z = x.clone()
    z[0, t[0]] = -math.inf  # pair 0's chosen sequence
    stats, _, seq, reward, dx = preference(z, t, bounds, ref, label_smoothing=smoothing)
    assert float(stats[0]) == math.inf and float(reward[0]) == -math.inf
    assert bool(torch.isfinite(dx).all()) and torch.equal(dx[4:], plain[4][4:])
    slope = -0.1 * (1 - smoothing) / pairs
    assert abs(float(dx[0, t[0]]) - slope) <= 4 * U * abs(slope)


@pytest.mark.parametrize("name, v", [("f16", (1 << 26) + 5), ("f32", 1 << 25)])
def test_sums_of_very_long_rows(name, v):
    """Equal terms that fp32 does not hold exactly: adding thousands of them up in fp32 rounds the same way
    again and again (6e-5 of the sum at 65,536 terms to a thread)."""
    up = float(torch.tensor(0.3).to(DT[name]))
    x = torch.zeros(2, v, dtype=DT[name], device=DEV)
    t = torch.tensor([v // 3, 7], device=DEV)
    x[0, t[0]] = up  # the target's own logit serves as the reference
    x[1, v // 2], x[1, 7] = up, -60.0  # the maximum has to
    rest = math.exp(-up)
    total = [1 + (v - 1) * rest, 1 + (v - 2) * rest + math.exp(-60.0 - up)]
    want = [-math.log(total[0]), -60.0 - up - math.log(total[1])]
    got = logprobs(x, t)
    for row in range(2):
        assert abs(float(got[row]) - want[row]) <= U * (2 * abs(want[row] + math.log(v)) + 2 + 26 + abs(want[row]))
    old = got - 0.1
    stats, lp, dx = policy(x, t, old, full(2, value=1.0))
    assert torch.equal(got, lp)
    ratio = math.exp(want[0] - float(old[0]))
    p = rest / total[0]
    e = 40 * U
    assert abs(float(dx[0, 0]) - ratio * p) <= ratio * p * (e + torch.finfo(DT[name]).eps / 2) + 2.0 ** -25


@pytest.mark.parametrize("v", [50, 3000, 140_000])
@pytest.mark.parametrize("n", [1, 24, 128])
def test_a_workspace_that_was_not_zero_shows(n, v):
    """The loss of few rows is formed by the last block to finish, which a count in the workspace names.  A count
    that does not start at 0 leaves NaN, never the values of an earlier call; the rest of the results hold."""
    x, t = grid_rows(n, v, 0.5, seed=10)
    adv, old = full(n, value=1.0), full(n, value=-2.0)
    want, logp, dx = policy(x, t, old, adv)
    for left in (0x0101010101010101, -1, 1, 23, 127):  # bytes, or the small numbers of some other tensor
        ws = zs.policy_workspace(n, DEV)
        ws[:ws.numel() // 8 * 8].view(torch.int64).fill_(left)
        stats, lp, d = full(4), full(n), torch.full_like(x, 5.0)
        for _ in range(2):  # nor does a second call with it
            zs.zero_policy_loss(x, t, old_logp=old, advantage=adv, divisor=1.0, stats=stats, logp=lp, dlogits=d,
                                workspace=ws)
            assert bool(torch.isnan(stats).all()), stats
            assert torch.equal(lp, logp) and torch.equal(d, dx)
    ws = zs.policy_workspace(n, DEV)
    for _ in range(3):
        zs.zero_policy_loss(x, t, old_logp=old, advantage=adv, divisor=1.0, stats=stats, logp=lp, dlogits=d, workspace=ws)
        assert torch.equal(stats, want)


def test_more_rows_need_no_count():
    """Past 128 rows a launch of its own adds up: any contents of the workspace will do."""
    x, t = grid_rows(129, 300, 0.5, seed=11)
    adv, old = full(129, value=1.0), full(129, value=-2.0)
    want, _, _ = policy(x, t, old, adv)
    stats, lp = full(4), full(129)
    zs.zero_policy_loss(x, t, old_logp=old, advantage=adv, divisor=1.0, stats=stats, logp=lp,
                        workspace=zs.policy_workspace(129, DEV).fill_(0xFF))
    assert torch.equal(stats, want)


def past_cache_rows(name, v):
    """Rows that are a little more than the 256 MB from which gradients are stored past the cache, and a slice of
    them that is less."""
    n = (1 << 28) // (v * torch.tensor([], dtype=DT[name]).element_size()) + 8
    g = torch.Generator(DEV).manual_seed(7)
    x = torch.empty(n, v, dtype=DT[name], device=DEV).normal_(0.0, 2.0, generator=g)
    t = torch.randint(0, v, (n,), generator=g, device=DEV)
    t[torch.rand(n, generator=g, device=DEV) < 0.1] = -100
    x[:, v - 3] = -math.inf
    t[t == v - 3] = 0
    return x, t


@pytest.mark.parametrize("name, v", [("f16", 50_001), ("bf16", 32_000), ("bf16", 131_080), ("f32", 8_000),
                                     ("f32", 131_079)])
def test_policy_gradient_past_the_cache(name, v):
    """A row's results do not depend on the others: the same bits as a call on the slice alone."""
    x, t = past_cache_rows(name, v)
    n, k = len(t), len(t) // 3
    g = torch.Generator(DEV).manual_seed(8)
    adv = torch.randn(n, generator=g, device=DEV)
    old = logprobs(x, t) + 0.2 * torch.randn(n, generator=g, device=DEV)
    _, logp, dx = policy(x, t, old, adv, ref=old, kl=0.1)
    for rows in (slice(0, k), slice(n - k, n)):
        _, lp, d = policy(x[rows], t[rows], old[rows], adv[rows], ref=old[rows], kl=0.1)
        assert torch.equal(lp, logp[rows]) and torch.equal(bits(d), bits(dx[rows]))
    assert int(dx[t < 0].count_nonzero()) == 0
    _, alone, _ = policy(x, t, old, adv, ref=old, kl=0.1, gradient=False)
    assert torch.equal(alone, logp)
    stats = policy(x, t, old, adv, ref=old, kl=0.1)[0], policy(x, t, old, adv, ref=old, kl=0.1, gradient=False)[0]
    assert torch.equal(*stats)


@pytest.mark.parametrize("name, v", [("f16", 50_001), ("bf16", 32_000), ("f32", 8_000), ("f32", 131_079)])
def test_preference_gradient_past_the_cache(name, v):
    """16 times the pairs of a slice at 16 times its gradient scale: the slice's rows have the same coefficients and
    with them the same bits."""
    x, t = past_cache_rows(name, v)
    n = len(t)
    few = 4
    pairs = 16 * few
    cuts = torch.linspace(0, n - 3, 2 * pairs + 1).long()
    cuts[2 * few] = max(2 * few, n // 3)  # the first pairs' rows are a third of all
    cuts[:2 * few] = torch.linspace(0, int(cuts[2 * few]) - 1, 2 * few + 1).long()[:2 * few]
    cuts = cuts.cummax(0).values.to(DEV)
    k = int(cuts[2 * few])
    ref = torch.linspace(-3000.0, -2990.0, 2 * pairs, device=DEV)
    every = preference(x, t, cuts, ref, grad_scale=16.0, beta=0.01)
    part = preference(x[:k], t[:k], cuts[:2 * few + 1], ref[:2 * few], grad_scale=1.0, beta=0.01)
    for i in (1, 2, 3):
        m = len(part[i])
        assert torch.equal(every[i][:m], part[i])
    assert torch.equal(bits(every[4][:k]), bits(part[4]))
    assert int(part[4].count_nonzero()) > 0 and bool(torch.isfinite(every[4]).all())
    assert int(every[4][n - 3:].count_nonzero()) == 0 and int(every[4][t < 0].count_nonzero()) == 0
    # the slice itself, by the definition
    lp, tol = exact_logp(x[:k], t[:k].clamp(min=0))
    counts = t[:k] >= 0
    assert bool(((part[1].double() - lp).abs() <= tol)[counts].all())
    sign = torch.zeros(k, dtype=torch.float64, device=DEV)
    h = (part[3][0::2] - part[3][1::2]).double()
    slope = 0.01 / few * (torch.sigmoid(h) - 1)
    for q in range(2 * few):
        sign[int(cuts[q]):int(cuts[q + 1])] = slope[q // 2] * (1 - 2 * (q % 2))
    coef = torch.where(counts, sign, 0.0)
    # h from rewards stored in fp32: u |reward| each, a quarter of it in sigmoid's slope
    e_h = U * part[3].double().abs().max() * 2
    for row in (0, 1, k // 2, k - 1):
        p = (x[row].double()).softmax(0)
        want = -coef[row] * p
        want[t[row].clamp(min=0)] += coef[row]
        spread = (x[row].double() - x[row, t[row].clamp(min=0)].double()).abs()
        e_p = U * (2 * torch.where(torch.isfinite(spread), spread, 0.0) + 6) + tol[row]
        err = coef[row].abs() * p * e_p + 0.01 / few * e_h + 4 * U * want.abs()
        err = err + (want.abs() + err) * torch.finfo(DT[name]).eps / 2 + (2.0 ** -25 if name == "f16" else 2.0 ** -126)
        assert bool(((part[4][row].double() - want).abs() <= err).all())


def test_many_pairs_without_a_gradient():
    """The launch for the pairs, only their statistics wanted."""
    x, t = grid_rows(100, 257, 0.5, seed=9)
    bounds = torch.arange(0, 101, 2, device=DEV)
    ref = torch.linspace(-30.0, -5.0, 50, device=DEV)
    a, b = preference(x, t, bounds, ref), preference(x, t, bounds, ref, gradient=False)
    for p, q in zip(a[:4], b[:4]):
        assert torch.equal(p, q)
    h = (a[3][0::2] - a[3][1::2]).double()
    assert abs(float(a[0][0]) + float(torch.nn.functional.logsigmoid(h).mean())) <= 1e-6
    assert float(a[0][1]) == float((h > 0).float().mean())
