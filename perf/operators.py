"""The post-training operators next to the owner-shard step, as measured cases.

Five kinds of call:

* ``step8``       one owner's Adam/AdamW step whose two moments are held in 8 bits
                  (``OwnerShard8.adam_step``), from rank gradients or a stored gradient;
* ``moments8``    the same moments brought from fp32 into 8 bits and back
                  (``OwnerShard8.pack_moments`` / ``unpack_moments``);
* ``logprobs``    log-probabilities of given tokens from logits (``zero_token_logprobs``);
* ``policy``      the clipped policy loss with a KL term, and its gradient of the logits
                  (``zero_policy_loss``);
* ``preference``  the paired log-ratio loss, and its gradient of the logits
                  (``zero_preference_loss``).

``run`` computes them in plain torch operations, or, where ``own`` is true, calls the library.
"""
import functools
import math
import random

import torch

own = False

BLOCK = 128          # elements that share one scale
E4M3_MAX = 448.0     # largest e4m3 value
E4M3_TINY = 2.0 ** -9  # smallest positive e4m3 value
TINY_MAX = 2.0 ** -100  # a block whose largest magnitude is below this holds zeros
HYPER = dict(lr=1e-3, beta1=0.8, beta2=0.999, eps=1e-8, weight_decay=3e-7, adamw=True)
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
LAYER = (4096 * 4096,) * 4 + (4096 * 11008,) * 3 + (4096,) * 2  # one decoder layer's tensors


def listed():
    step = dict(kind="step8", align=64, step=11, clip=1.0)
    return [
        # the smallest call: the owner of three short tensors, where the launch is all there is
        dict(step, name="step8 three tensors", tensors="three", ranks=4, owner=1, grad="f16", param="f16"),
        # many tensors of 100 elements padded to 128 (biases, norms): every block holds padding
        dict(step, name="step8 ragged", tensors="equal", count=200_000, numel=100, ranks=4, owner=1, grad="f16",
             param="f16"),
        # four decoder layers over eight ranks, the owner cut inside its tensors
        dict(step, name="step8 four layers", tensors="layers", count=4, ranks=8, owner=1, grad="bf16", param="bf16"),
        # the second pass of a checked step: a quarter of 1.5e9 elements from the stored fp32 gradient, clipped
        dict(step, name="step8 stored gradient", tensors="equal", count=1, numel=1_500_000_000, ranks=4, owner=1,
             grad="stored", param="f16", clip=0.25),
        # a resumed 32-bit checkpoint goes over to 8 bits
        dict(kind="moments8", name="moments8 pack layers", direction="pack", tensors="layers", count=4, ranks=8,
             owner=1, align=64),
        # an 8-bit state leaves for a checkpoint in fp32, small padded tensors
        dict(kind="moments8", name="moments8 unpack ragged", direction="unpack", tensors="equal", count=200_000,
             numel=100, ranks=4, owner=1, align=64),
        # scoring one token as it is generated
        dict(kind="logprobs", name="logprobs one token", rows=1, vocab=32_000, dtype="bf16", temperature=1.0),
        # the reference model's pass over a batch of 4096 tokens, large vocabulary
        dict(kind="logprobs", name="logprobs batch", rows=4096, vocab=128_000, dtype="bf16", temperature=1.0),
        # a short answer in half precision, an odd vocabulary: rows start at any 2-byte address
        dict(kind="policy", name="policy short odd", rows=24, vocab=50_001, dtype="f16", temperature=0.7,
             kl_coef=0.05),
        # one policy update's micro batch: 8192 tokens, large vocabulary
        dict(kind="policy", name="policy batch", rows=8192, vocab=128_000, dtype="bf16", temperature=1.0,
             kl_coef=0.02),
        # two short pairs in fp32
        dict(kind="preference", name="preference two pairs", pairs=2, shortest=3, longest=17, vocab=1000, dtype="f32",
             average=False),
        # eight pairs of up to 768 tokens
        dict(kind="preference", name="preference batch", pairs=8, shortest=256, longest=768, vocab=32_000,
             dtype="bf16", average=False),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    kind = rng.choice(["step8", "moments8", "logprobs", "policy", "preference"])
    if kind in ("step8", "moments8"):
        ranks = rng.choice([1, 2, 3, 4, 5, 8])
        owned = _spread(rng, 500, 60_000_000)
        if rng.random() < 0.5:  # one flat run
            shape = dict(tensors="equal", count=1, numel=owned * ranks + rng.randrange(97))
        else:  # tensors of any length, most with padding after them
            numel = _spread(rng, 1, min(owned, 100_000))
            shape = dict(tensors="equal", count=max(1, min(100_000, owned * ranks // numel)), numel=numel)
        case = dict(kind=kind, **shape, ranks=ranks, owner=rng.randrange(ranks), align=rng.choice([1, 8, 64, 128]))
        if kind == "moments8":
            return dict(case, direction=rng.choice(["pack", "unpack"]))
        return dict(case, grad=rng.choice(["f16", "bf16", "f32", "stored"]), param=rng.choice(["f16", "bf16", "none"]),
                    step=rng.randrange(1, 2000), clip=rng.choice([1.0, 0.37]))
    dtype = rng.choice(["f16", "bf16", "f32"])
    vocab = _spread(rng, 200, 131_072)
    most = 150_000_000 // vocab  # logits of one call
    if kind == "preference":
        pairs = _spread(rng, 1, 16)
        longest = _spread(rng, 2, max(2, min(600, most // (2 * pairs))))
        return dict(kind=kind, pairs=pairs, shortest=rng.randrange(1, longest + 1), longest=longest, vocab=vocab,
                    dtype=dtype, average=rng.random() < 0.3)
    case = dict(kind=kind, rows=_spread(rng, 1, min(8192, most)), vocab=vocab, dtype=dtype,
                temperature=rng.choice([1.0, 0.7, 1.3]))
    return dict(case, kl_coef=rng.choice([0.0, 0.02, 0.1])) if kind == "policy" else case


# ---------------------------------------------------------------- sizes
def _layout(case):
    """(tensor sizes, begin, end, base, blocks): tensors padded to `align` one after another, owner r of R holding
    [P r / R, P (r + 1) / R) of the padded total P; owner-local arrays start at `base` and hold whole blocks."""
    if case["tensors"] == "three":
        numels = [1000, 37, 5003]
    elif case["tensors"] == "layers":
        numels = list(LAYER) * case["count"]
    else:
        numels = [case["numel"]] * case["count"]
    a = case["align"]
    total = sum(-(-n // a) * a for n in numels)
    begin = total * case["owner"] // case["ranks"]
    end = total * (case["owner"] + 1) // case["ranks"]
    base = begin // BLOCK * BLOCK
    return numels, begin, end, base, -(-(end - base) // BLOCK)


def _real_count(case):
    numels, begin, end, _, _ = _layout(case)
    a, at, count = case["align"], 0, 0
    for n in numels:
        count += max(0, min(end, at + n) - max(begin, at))
        at += -(-n // a) * a
    return count


def _lengths(case):
    """Token counts of the 2 * pairs sequences: chosen, rejected, chosen, ..."""
    span = case["longest"] - case["shortest"] + 1
    return [case["shortest"] + (i * 7919 + 11) % span for i in range(2 * case["pairs"])]


def _rows(case):
    return sum(_lengths(case)) if case["kind"] == "preference" else case["rows"]


def work(case):
    kind = case["kind"]
    if kind in ("step8", "moments8"):
        n = _real_count(case)
        scales = 2 * 4 / BLOCK
        if kind == "moments8":
            return {"bytes": n * (8 + 2 + scales), "flops": n * 8}
        grad = 4 if case["grad"] == "stored" else case["ranks"] * SIZE[case["grad"]]
        param = 0 if case["param"] == "none" else 2
        # master read and written, two 8-bit moments and their scales read and written
        return {"bytes": n * (grad + 8 + 4 + 2 * scales + param), "flops": n * (32 + case["ranks"])}
    n, logits = _rows(case), _rows(case) * case["vocab"] * SIZE[case["dtype"]]
    if kind == "logprobs":
        return {"bytes": logits + n * (8 + 4), "flops": 4 * n * case["vocab"]}
    per_row = 8 + 4 + (16 if kind == "policy" else 0)
    return {"bytes": 2 * logits + n * per_row, "flops": 7 * n * case["vocab"]}


# ---------------------------------------------------------------- inputs
def _encode(x, positive):
    """A whole number of blocks in 8 bits: (codes as float8_e4m3fn, one scale a block)."""
    b = x.view(-1, BLOCK)
    top = b.abs().amax(1, keepdim=True)
    live = top >= TINY_MAX
    inv = torch.where(live, E4M3_MAX / top, torch.zeros_like(top))
    q = b * inv
    if positive:  # what is above zero stays above zero
        q = torch.where((b > 0) & live, q.clamp_min(E4M3_TINY), q)
    scale = torch.where(live, top / E4M3_MAX, torch.zeros_like(top))
    return q.to(torch.float8_e4m3fn).view(-1), scale.view(-1)


def _decode(codes, scale):
    return (codes.float().view(-1, BLOCK) * scale.view(-1, 1)).view(-1)


def _prepare_owner(case, seed):
    numels, begin, end, base, blocks = _layout(case)
    dev, n, a = "cuda", blocks * BLOCK, case["align"]
    gen = torch.Generator(dev).manual_seed(seed)
    rand = functools.partial(torch.randn, n, generator=gen, device=dev)
    # which elements of [base, base + n) are the owner's own and belong to a tensor
    f = torch.arange(base, base + n, device=dev)
    real = (f >= begin) & (f < end)
    if case["tensors"] == "equal":
        pitch = -(-case["numel"] // a) * a
        real &= f % pitch < case["numel"]
    elif case["tensors"] == "three":
        pad, at = [], 0
        for m in numels:
            pad.append((at + m, -(-(at + m) // a) * a))
            at = pad[-1][1]
        for lo, hi in pad:
            real &= (f < lo) | (f >= hi)
    del f  # a decoder layer's tensors are whole multiples of the alignment
    s = {"case": case, "real": real, "base": base, "all_real": bool(real.all())}
    hold = lambda x: x.masked_fill_(~real, 0)  # noqa: E731
    # moments as a run some steps old leaves them: roots of the second moment spread over a decade
    m = hold(rand() * 2e-4)
    r = hold((rand() * 0.8).exp_() * 4e-4)
    if case["kind"] == "moments8":
        s["m"], s["v"] = m, r.square_()
        if case["direction"] == "unpack":
            s["m8"], s["ms"] = _encode(s["m"], False)
            s["r8"], s["rs"] = _encode(s["v"].sqrt(), True)
        else:
            s["m8"], s["r8"] = (torch.zeros(n, dtype=torch.float8_e4m3fn, device=dev) for _ in range(2))
            s["ms"], s["rs"] = (torch.zeros(blocks, device=dev) for _ in range(2))
    else:
        s["m8"], s["ms"] = _encode(m, False)
        s["r8"], s["rs"] = _encode(r, True)
        del m, r
        s["w"] = hold(rand() * 0.02)
        if case["grad"] == "stored":
            s["g"] = hold(rand() * 1e-3)
        else:
            s["grads"] = [hold(rand() * 1e-3).to(DTYPES[case["grad"]]) for _ in range(case["ranks"])]
        s["p16"] = None if case["param"] == "none" else torch.zeros(n, dtype=DTYPES[case["param"]], device=dev)
    if own:  # the plan that a program makes once: layout, table of pieces, state
        import zero_sharded_optimizer_owned_amd as zs

        sh = s["shard"] = zs.OwnerShard8(numels, case["ranks"], case["owner"], align=a, device=dev)
        sh.exp_avg8, sh.exp_avg_scale, sh.exp_rms8, sh.exp_rms_scale = s["m8"], s["ms"], s["r8"], s["rs"]
        if case["kind"] == "step8":
            sh.master = s["w"]
    return s


def _prepare_tokens(case, seed):
    dev, n, v = "cuda", _rows(case), case["vocab"]
    gen = torch.Generator(dev).manual_seed(seed)
    rows = torch.arange(n, device=dev)
    said = v - v // 64  # the columns after these only pad the vocabulary: no token has them
    targets = torch.randint(0, said, (n,), generator=gen, device=dev)
    logits = torch.empty(n, v, dtype=DTYPES[case["dtype"]], device=dev)
    logits.normal_(0.0, 2.0, generator=gen)
    logits[:, said:] = -math.inf
    # what was said is mostly likely
    logits[rows, targets] += (7.0 + 2.0 * torch.randn(n, generator=gen, device=dev)).to(logits.dtype)
    # prompt and padding positions count for nothing
    skip = torch.rand(n, generator=gen, device=dev) < 0.15
    skip[0] = False
    targets.masked_fill_(skip, -100)
    s = {"case": case, "logits": logits, "targets": targets, "logp": torch.empty(n, device=dev)}
    if case["kind"] == "logprobs":
        return s
    s["dlogits"] = torch.empty_like(logits)
    s["grad_scale"] = 1024.0 if case["dtype"] == "f16" else 1.0  # half precision: a loss scale
    t = case.get("temperature", 1.0)
    lp = torch.empty(n, dtype=torch.float64, device=dev)
    at = targets.clamp_min(0)
    for i in range(0, n, 1024):
        x = logits[i:i + 1024].double() / t
        lp[i:i + 1024] = x.gather(1, at[i:i + 1024, None])[:, 0] - x.logsumexp(1)
    noise = lambda k, sd: torch.randn(k, generator=gen, device=dev, dtype=torch.float64) * sd  # noqa: E731
    if case["kind"] == "policy":
        d = noise(n, 0.15)  # log ratio to the policy that sampled, some beyond the clip borders
        for border in (math.log(0.8), math.log(1.28)):  # at a border, rounding alone would choose the side
            near = (d - border).abs() < 2e-3
            d = torch.where(near, d + torch.where(d >= border, 4e-3, -4e-3), d)
        s["old_logp"] = (lp - d).float()
        s["ref_logp"] = (lp + noise(n, 0.2)).float()
        s["advantage"] = torch.randn(n, generator=gen, device=dev)
        # answers of 1 to 64 tokens, each weighted by its length
        s["weight"] = 1.0 / torch.randint(1, 65, (n,), generator=gen, device=dev).float()
        s["divisor"] = float(max(1, n // 16))
        s["stats"] = torch.empty(4, device=dev)
    else:
        lens = _lengths(case)
        ends = torch.tensor([0] + lens).cumsum(0)
        s["seq_begin"] = ends.to(dev)
        sums = torch.zeros(len(lens), dtype=torch.float64, device=dev)
        of = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).to(dev)
        sums.index_add_(0, of, torch.where(targets >= 0, lp, torch.zeros_like(lp)))
        s["seq_of"], s["beta"], s["smoothing"] = of, 0.1, 0.05
        s["ref_logp"] = (sums + noise(len(lens), 6.0)).float()  # the reference model's sums
        s["seq_logp"], s["reward"] = (torch.empty(len(lens), device=dev) for _ in range(2))
        s["stats"] = torch.empty(2, device=dev)
    if own:
        import zero_sharded_optimizer_owned_amd as zs

        s["workspace"] = (zs.policy_workspace(n, dev) if case["kind"] == "policy"
                          else zs.preference_workspace(n, case["pairs"], dev))
    return s


def prepare(case, seed):
    return (_prepare_owner if case["kind"] in ("step8", "moments8") else _prepare_tokens)(case, seed)


# ---------------------------------------------------------------- the plain forms
def _plain_step(s):
    c, h = s["case"], HYPER
    if c["grad"] == "stored":
        g = s["g"]
    else:
        g = functools.reduce(lambda x, y: x + y.float(), s["grads"], torch.zeros_like(s["w"])) / c["ranks"]
    g = g * c["clip"]
    w, r = s["w"], _decode(s["r8"], s["rs"])
    m = h["beta1"] * _decode(s["m8"], s["ms"]) + (1 - h["beta1"]) * g
    v = h["beta2"] * r * r + (1 - h["beta2"]) * g * g
    r = v.sqrt()
    step_size = h["lr"] / (1 - h["beta1"] ** c["step"])
    denom = r * (1 / math.sqrt(1 - h["beta2"] ** c["step"])) + h["eps"]
    new = w * (1 - h["lr"] * h["weight_decay"]) - step_size * (m / denom)
    if not s["all_real"]:
        zero = torch.zeros_like(w)
        new, m, r = (torch.where(s["real"], x, y) for x, y in ((new, w), (m, zero), (r, zero)))
    w.copy_(new)
    m8, ms = _encode(m, False)
    r8, rs = _encode(r, True)
    for k, x in (("m8", m8), ("ms", ms), ("r8", r8), ("rs", rs)):
        s[k].copy_(x)
    if s["p16"] is not None:
        s["p16"].copy_(new.to(s["p16"].dtype))
    return _owner_outputs(s)


def _owner_outputs(s):
    keys = ("w", "m8", "ms", "r8", "rs", "p16")
    return {k: s[k] for k in keys if s[k] is not None}


def _plain_moments(s):
    if s["case"]["direction"] == "pack":
        s["m8"], s["ms"] = _encode(s["m"], False)
        s["r8"], s["rs"] = _encode(s["v"].sqrt(), True)
        return {k: s[k] for k in ("m8", "ms", "r8", "rs")}
    s["m"].copy_(_decode(s["m8"], s["ms"]))
    s["v"].copy_(_decode(s["r8"], s["rs"]).square())
    return {"m": s["m"], "v": s["v"]}


def _plain_rows(logits, targets, temperature):
    """(probabilities, log-probability of the target or 0, whether the row counts, target or 0).  Elements in fp32; a
    row's sum and its logarithm in fp64, since hundreds of tokens' errors of one sign add up in a sequence."""
    x = logits.float() / temperature
    top = x.amax(1, keepdim=True)
    x = x - torch.where(top == -math.inf, 0.0, top)
    e = x.exp()
    total = e.sum(1, keepdim=True, dtype=torch.float64)
    counts = (targets >= 0) & (targets < logits.shape[1]) & (total[:, 0] != 0)
    at = torch.where(counts, targets, 0)
    lp = x.gather(1, at[:, None])[:, 0].double() - total[:, 0].log()
    return e * (1 / total).float(), torch.where(counts, lp, 0.0), counts, at


def _plain_grad(p, at, coef, dtype):
    """coef * (one at the target - p), rows of no weight zero."""
    d = torch.where(coef[:, None] != 0, p * -coef[:, None], 0.0)
    d[torch.arange(len(at), device=at.device), at] += coef
    return d.to(dtype)


def _plain_logprobs(s):
    _, lp, _, _ = _plain_rows(s["logits"], s["targets"], s["case"]["temperature"])
    return {"logp": lp.float()}


def _plain_policy(s):
    c = s["case"]
    p, lp, counts, at = _plain_rows(s["logits"], s["targets"], c["temperature"])
    weight = torch.where(counts, s["weight"], 0.0) / s["divisor"]
    a, ratio = s["advantage"], (lp - s["old_logp"]).exp()
    free, held = a * ratio, a * ratio.clamp(0.8, 1.28)
    inside = free <= held
    d = s["ref_logp"] - lp
    kl = d.exp() - d - 1
    parts = [(weight * x).sum() for x in (-torch.where(inside, free, held), kl, (~inside).double())]
    stats = torch.stack([parts[0] + c["kl_coef"] * parts[1], *parts]).float()
    slope = torch.where(inside, -free, 0.0) + c["kl_coef"] * (1 - d.exp())
    coef = torch.where(counts, weight * slope * (s["grad_scale"] / c["temperature"]), 0.0).float()
    return {"stats": stats, "logp": lp.float(), "dlogits": _plain_grad(p, at, coef, s["logits"].dtype)}


def _plain_preference(s):
    c, beta, eps = s["case"], s["beta"], s["smoothing"]
    p, lp, counts, at = _plain_rows(s["logits"], s["targets"], 1.0)
    zero = torch.zeros(2 * c["pairs"], dtype=torch.float64, device=lp.device)
    sums, tokens = zero.index_add(0, s["seq_of"], lp), zero.index_add(0, s["seq_of"], counts.double())
    part = 1.0 / tokens.clamp_min(1) if c["average"] else torch.ones_like(tokens)
    seq = sums * part
    reward = beta * (seq - s["ref_logp"].double() * part)
    h = reward[0::2] - reward[1::2]
    softplus = lambda x: x.clamp_min(0) + (-x.abs()).exp().log1p()  # noqa: E731
    loss = ((1 - eps) * softplus(-h) + eps * softplus(h)).mean()
    share = (h > 0).double().mean()
    # d loss / d h, then down to each sequence's tokens
    slope = (eps / (1 + (-h).exp()) - (1 - eps) / (1 + h.exp())) * beta / c["pairs"]
    coef = (torch.stack([slope, -slope], 1).view(-1) * part * s["grad_scale"])[s["seq_of"]]
    coef = torch.where(counts, coef, 0.0).float()
    return {"stats": torch.stack([loss, share]).float(), "logp": lp.float(), "seq_logp": seq.float(),
            "reward": reward.float(), "dlogits": _plain_grad(p, at, coef, s["logits"].dtype)}


# ---------------------------------------------------------------- the library's calls
def _own_step(s):
    c, sh = s["case"], s["shard"]
    source = {"reduced_g": s["g"]} if c["grad"] == "stored" else {"rank_grads": s["grads"], "grad_base": s["base"],
                                                                  "divisor": float(c["ranks"])}
    sh.adam_step(step=c["step"], hyper=HYPER, param16=s["p16"], param_base=s["base"], clip_coef=c["clip"], **source)
    return _owner_outputs(s)


def _own_moments(s):
    if s["case"]["direction"] == "pack":
        s["shard"].pack_moments(s["m"], s["v"])
        return {k: s[k] for k in ("m8", "ms", "r8", "rs")}
    s["shard"].unpack_moments(s["m"], s["v"])
    return {"m": s["m"], "v": s["v"]}


def _own_logprobs(s):
    import zero_sharded_optimizer_owned_amd as zs

    zs.zero_token_logprobs(s["logits"], s["targets"], s["logp"], temperature=s["case"]["temperature"])
    return {"logp": s["logp"]}


def _own_policy(s):
    import zero_sharded_optimizer_owned_amd as zs

    c = s["case"]
    zs.zero_policy_loss(s["logits"], s["targets"], old_logp=s["old_logp"], ref_logp=s["ref_logp"],
                        advantage=s["advantage"], weight=s["weight"], divisor=s["divisor"], clip_low=0.2,
                        clip_high=0.28, kl_coef=c["kl_coef"], temperature=c["temperature"],
                        grad_scale=s["grad_scale"], stats=s["stats"], logp=s["logp"], dlogits=s["dlogits"],
                        workspace=s["workspace"])
    return {k: s[k] for k in ("stats", "logp", "dlogits")}


def _own_preference(s):
    import zero_sharded_optimizer_owned_amd as zs

    zs.zero_preference_loss(s["logits"], s["targets"], s["seq_begin"], ref_logp=s["ref_logp"], beta=s["beta"],
                            label_smoothing=s["smoothing"], average=s["case"]["average"],
                            grad_scale=s["grad_scale"], stats=s["stats"], logp=s["logp"], seq_logp=s["seq_logp"],
                            reward=s["reward"], dlogits=s["dlogits"], workspace=s["workspace"])
    return {k: s[k] for k in ("stats", "logp", "seq_logp", "reward", "dlogits")}


PLAIN = dict(step8=_plain_step, moments8=_plain_moments, logprobs=_plain_logprobs, policy=_plain_policy,
             preference=_plain_preference)
OWN = dict(step8=_own_step, moments8=_own_moments, logprobs=_own_logprobs, policy=_own_policy,
           preference=_own_preference)


def run(state):
    return (OWN if own else PLAIN)[state["case"]["kind"]](state)


# ---------------------------------------------------------------- the definitions, in 64 bits
def _round_e4m3(x):
    """Nearest e4m3 value (ties to even) of numbers up to 464: 3 bits below the leading one, steps of 2^-9 below 2^-6."""
    step = torch.exp2(torch.frexp(x)[1].clamp_min(-5).double() - 4)
    return torch.round(x / step) * step


def _exact_blocks(x, positive):
    b = x.view(-1, BLOCK)
    top = b.abs().max(1, keepdim=True).values
    top = torch.where(top < TINY_MAX, math.inf, top)  # the whole block is zero then
    q = _round_e4m3(b * E4M3_MAX / top)
    if positive:
        q = torch.where((b > 0) & (q == 0) & torch.isfinite(top), E4M3_TINY, q)
    return q.view(-1), torch.where(torch.isfinite(top), top / E4M3_MAX, 0.0).view(-1)


def _exact_owner(case, seed):
    s = _prepare_owner(case, seed)
    spread = lambda k: s[k].double().repeat_interleave(BLOCK)  # noqa: E731
    if case["kind"] == "moments8":
        if case["direction"] == "unpack":
            return {"m": s["m8"].double() * spread("ms"), "v": (s["r8"].double() * spread("rs")) ** 2}
        out = {}
        out["m8"], out["ms"] = _exact_blocks(s["m"].double(), False)
        out["r8"], out["rs"] = _exact_blocks(s["v"].double() ** 0.5, True)
        return out
    h, t = HYPER, case["step"]
    if case["grad"] == "stored":
        g = s["g"].double()
    else:
        g = torch.zeros_like(s["w"], dtype=torch.float64)
        for x in s["grads"]:
            g += x
        g /= case["ranks"]
    g = g.mul_(case["clip"]) * s["real"]
    m = s["m8"].double() * spread("ms") * h["beta1"] + (1 - h["beta1"]) * g
    v = (s["r8"].double() * spread("rs")) ** 2 * h["beta2"] + (1 - h["beta2"]) * g ** 2
    del g
    hat = (m / (1 - h["beta1"] ** t)) / ((v / (1 - h["beta2"] ** t)) ** 0.5 + h["eps"])
    w = s["w"].double()
    w = w - s["real"] * (h["lr"] * h["weight_decay"] * w + h["lr"] * hat)
    out = {"w": w}
    if s["p16"] is not None:
        out["p16"] = w
    out["m8"], out["ms"] = _exact_blocks(m * s["real"], False)
    out["r8"], out["rs"] = _exact_blocks(v ** 0.5 * s["real"], True)
    return out


def _exact_tokens(case, seed):
    s = _prepare_tokens(case, seed)
    t = case.get("temperature", 1.0)
    scored = s["targets"] >= 0
    rows, at = torch.arange(len(scored), device="cuda")[scored], s["targets"][scored]
    table = torch.log_softmax(s["logits"].double() / t, 1)
    lp = torch.zeros(len(scored), dtype=torch.float64, device="cuda")
    lp[rows] = table[rows, at]
    out = {"logp": lp}
    if case["kind"] == "logprobs":
        return out
    slope = torch.zeros_like(lp)  # of the loss, by each token's log-probability
    if case["kind"] == "policy":
        share = s["weight"].double() / s["divisor"] * scored
        a, ratio = s["advantage"].double(), torch.exp(lp - s["old_logp"].double())
        gain = torch.minimum(a * ratio, a * torch.clip(ratio, 0.8, 1.28))
        clipped = gain < a * ratio
        log_q = s["ref_logp"].double() - lp
        kl = torch.expm1(log_q) - log_q
        sums = [-(share * gain).sum(), (share * kl).sum(), (share * clipped).sum()]
        out["stats"] = torch.stack([sums[0] + case["kl_coef"] * sums[1], *sums])
        slope = share * (-(a * ratio) * ~clipped - case["kl_coef"] * torch.expm1(log_q)) / t
    else:
        lens, beta, eps = _lengths(case), s["beta"], s["smoothing"]
        parts = [x[y] for x, y in zip(lp.split(lens), scored.split(lens))]
        div = [max(1, len(x)) if case["average"] else 1 for x in parts]
        seq = torch.stack([x.sum() / d for x, d in zip(parts, div)])
        ref = s["ref_logp"].double() / torch.tensor(div, device="cuda", dtype=torch.float64)
        out["seq_logp"], out["reward"] = seq, beta * (seq - ref)
        h = out["reward"].view(-1, 2) @ torch.tensor([1.0, -1.0], dtype=torch.float64, device="cuda")
        loss = -(1 - eps) * torch.nn.functional.logsigmoid(h) - eps * torch.nn.functional.logsigmoid(-h)
        out["stats"] = torch.stack([loss.mean(), (h > 0).double().mean()])
        per_pair = beta / case["pairs"] * (torch.sigmoid(h) - (1 - eps))
        of = s["seq_of"]
        sign = 1.0 - 2.0 * (of % 2).double()
        slope = per_pair[of // 2] * sign / torch.tensor(div, device="cuda", dtype=torch.float64)[of] * scored
    slope = slope * s["grad_scale"]
    grad = table.exp_().mul_(-slope[:, None])
    grad[rows, at] += slope[rows]
    out["dlogits"] = grad
    return out


def exact(case, seed):
    return (_exact_owner if case["kind"] in ("step8", "moments8") else _exact_tokens)(case, seed)
