"""The operators at the model's two ends, and of what its backward pass keeps, as measured cases.

Five kinds of call:

* ``embed``       embedding lookup with scaling (``zero_embedding``);
* ``embed_grad``  its gradient, sums over equal tokens in a fixed order (``zero_embedding_grad``);
* ``norm``        root-mean-square norm with the residual's addition, and the residual stream kept in 8 bits
                  for the backward pass (``zero_rms_norm``);
* ``norm_grad``   its backward pass from the 16-bit or the 8-bit residual stream
                  (``zero_rms_norm_restore``, ``zero_rms_norm_backward``);
* ``head``        softmax cross entropy straight from hidden states and the output weights, with its gradients
                  of both, the logits of a bounded number of rows at a time (``zero_linear_cross_entropy``).

``run`` computes them in plain torch operations, or, where ``own`` is true, calls the library.
"""
import math

import torch

own = False

BLOCK = 128        # elements of a row that share one scale
E4M3_MAX = 448.0   # largest e4m3 value
TINY_MAX = 2.0 ** -100  # a block whose largest magnitude is below this holds zeros
EPS = 1e-6
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}


def listed():
    return [
        # one token enters the model as it is generated: the launch is all there is
        dict(kind="embed", name="embed one token", tokens=1, vocab=32_000, dim=4096, dtype="bf16"),
        # a training batch of 16,384 tokens, large vocabulary
        dict(kind="embed", name="embed batch", tokens=16_384, vocab=128_000, dim=4096, dtype="bf16"),
        # a short batch added onto the gradient that the output head left in a tied table, odd sizes
        dict(kind="embed_grad", name="embed_grad short tied", tokens=333, vocab=50_001, dim=1000, dtype="f16",
             accumulate=True),
        # a training batch's whole gradient: most rows of the table are zero, a few tokens are very frequent
        dict(kind="embed_grad", name="embed_grad batch", tokens=16_384, vocab=128_000, dim=4096, dtype="bf16",
             accumulate=False),
        # four tokens generated at a time
        dict(kind="norm", name="norm four rows", rows=4, dim=4096, dtype="bf16", residual=True, keep=False),
        # a training batch that keeps its residual stream in 8 bits
        dict(kind="norm", name="norm batch kept", rows=16_384, dim=4096, dtype="bf16", residual=True, keep=True),
        # an odd width in half precision, from the 16-bit residual stream
        dict(kind="norm_grad", name="norm_grad odd", rows=999, dim=5003, dtype="f16", keep=False, upstream=False),
        # the batch's backward pass from 8 bits: the next product's input again, then the gradients
        dict(kind="norm_grad", name="norm_grad batch kept", rows=16_384, dim=4096, dtype="bf16", keep=True,
             upstream=True),
        # scoring one token as it is generated
        dict(kind="head", name="head one token", rows=1, vocab=32_000, dim=4096, dtype="bf16", grad=False,
             temperature=1.0, weighted=False),
        # a short answer in half precision with a loss scale, odd vocabulary
        dict(kind="head", name="head short odd", rows=77, vocab=50_001, dim=1000, dtype="f16", grad=True,
             temperature=0.7, weighted=True),
        # the reference model scores a batch, large vocabulary
        dict(kind="head", name="head score batch", rows=4096, vocab=128_000, dim=4096, dtype="bf16", grad=False,
             temperature=1.0, weighted=False),
        # a training step's loss and gradients, large vocabulary
        dict(kind="head", name="head train batch", rows=8192, vocab=128_000, dim=4096, dtype="bf16", grad=True,
             temperature=1.0, weighted=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    kind = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "head"])
    dtype = rng.choice(["f16", "bf16", "f32"])
    if kind in ("embed", "embed_grad"):
        dim = _spread(rng, 1, 8192)
        case = dict(kind=kind, tokens=_spread(rng, 1, min(60_000, 80_000_000 // dim)),
                    vocab=_spread(rng, 200, min(131_072, 400_000_000 // dim)), dim=dim, dtype=dtype)
        return dict(case, accumulate=rng.random() < 0.5) if kind == "embed_grad" else case
    if kind in ("norm", "norm_grad"):
        dim = _spread(rng, 1, 16_384)
        case = dict(kind=kind, rows=_spread(rng, 1, min(60_000, 80_000_000 // dim)), dim=dim, dtype=dtype,
                    keep=rng.random() < 0.5)
        return dict(case, **{"residual" if kind == "norm" else "upstream": rng.random() < 0.7})
    dim, vocab = 8 * _spread(rng, 1, 1024), _spread(rng, 200, 131_072)
    most = 600_000_000_000 // (vocab * dim)  # products of one call
    return dict(kind=kind, rows=_spread(rng, 1, max(1, min(6000, most, 400_000_000 // vocab))), vocab=vocab, dim=dim,
                dtype=rng.choice(["f16", "bf16"]), grad=rng.random() < 0.7, temperature=rng.choice([1.0, 0.7, 1.3]),
                weighted=rng.random() < 0.5)


def _scales(dim):
    return -(-dim // BLOCK)


def _ignored(rows):
    """Which rows count for nothing (prompt, padding): 3 in 20, never the first."""
    i = torch.arange(rows)
    return ((i * 7919 + 11) % 20 < 3) & (i > 0)


def work(case):
    b, kind, d = SIZE[case["dtype"]], case["kind"], case["dim"]
    if kind == "embed":
        n = case["tokens"] * d
        return {"bytes": 2 * b * n + 8 * case["tokens"], "flops": n}
    if kind == "embed_grad":
        n = case["tokens"] * d
        # the whole gradient is written; added onto another one, the rows of the tokens are read and written,
        # of which there are at most as many as tokens
        rows = 2 * min(case["tokens"], case["vocab"]) if case["accumulate"] else case["vocab"]
        return {"bytes": b * n + 8 * case["tokens"] + b * rows * d, "flops": 2 * n}
    if kind == "norm":
        n = case["rows"] * d
        moved = b * n * (2 + 2 * case["residual"])  # x and y; the residual and the sum
        if case["keep"]:
            moved += n + 4 * case["rows"] * _scales(d)
        return {"bytes": moved + 4 * case["rows"] + b * d, "flops": n * (5 + 2 * case["keep"])}
    if kind == "norm_grad":
        n = case["rows"] * d
        held = n + 4 * case["rows"] * _scales(d) if case["keep"] else b * n
        moved = held + b * n * (2 + case["upstream"] + case["keep"])  # dy, dx; its residual's part; y again
        return {"bytes": moved + 4 * case["rows"] + 2 * b * d, "flops": n * 10}
    live = case["rows"] - int(_ignored(case["rows"]).sum())
    both = (live + case["vocab"]) * d * b  # hidden states and weights, or their gradients
    rows = case["rows"]
    return {"bytes": both * (2 if case["grad"] else 1) + rows * (12 + 4 * case["weighted"]),
            "flops": 2 * live * case["vocab"] * d * (3 if case["grad"] else 1)}


# ---------------------------------------------------------------- inputs
def _tokens(case, gen):
    """Token numbers as text has them: frequency falls with the rank; some positions are padding."""
    n, v = case["tokens"], case["vocab"]
    rank = torch.exp(torch.rand(n, generator=gen, device="cuda", dtype=torch.float64) * math.log(v + 1)).long() - 1
    order = torch.randperm(v, generator=gen, device="cuda")
    tokens = order[rank.clamp(0, v - 1)]
    pad = torch.rand(n, generator=gen, device="cuda") < 0.03
    pad[0] = False
    return tokens.masked_fill_(pad, -1)


def _encode(x):
    """Rows in 8 bits: (codes as float8_e4m3fn, one scale for each block of a row)."""
    n, d = x.shape
    pad = _scales(d) * BLOCK - d
    b = torch.nn.functional.pad(x, (0, pad)).view(n, -1, BLOCK)
    top = b.abs().amax(2, keepdim=True)
    live = top >= TINY_MAX
    inv = torch.where(live, E4M3_MAX / top, torch.zeros_like(top))
    codes = (b * inv).to(torch.float8_e4m3fn).view(n, -1)[:, :d].contiguous()
    return codes, torch.where(live, top / E4M3_MAX, torch.zeros_like(top)).view(n, -1)


def _decode(codes, scale):
    return codes.float() * scale.repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def prepare(case, seed):
    dev, kind, d, dt = "cuda", case["kind"], case["dim"], DTYPES[case["dtype"]]
    gen = torch.Generator(dev).manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device=dev)  # noqa: E731
    s = {"case": case}
    if kind in ("embed", "embed_grad"):
        n, v = case["tokens"], case["vocab"]
        s["tokens"], s["scale"] = _tokens(case, gen), math.sqrt(d)
        if kind == "embed":
            s["table"] = torch.empty(v, d, dtype=dt, device=dev).normal_(0, 0.02, generator=gen)
            s["out"] = torch.empty(n, d, dtype=dt, device=dev)
            return s
        s["dout"] = (rand(n, d) * 0.01).to(dt)
        s["dtable"] = torch.empty(v, d, dtype=dt, device=dev)
        if case["accumulate"]:
            s["dtable"].normal_(0, 0.1, generator=gen)
        if own:
            import zero_sharded_optimizer_owned_amd as zs

            s["workspace"] = zs.embedding_workspace(n, v, d, dev)
        return s
    n = case["rows"]
    if kind in ("norm", "norm_grad"):
        s["gain"] = (1 + 0.2 * rand(d)).to(dt)
        # a residual stream: a few channels are much larger than the rest
        channel = torch.where(torch.rand(d, generator=gen, device=dev) < 0.01, 20.0, 1.0)
        h = (rand(n, d) * channel).to(dt)
        if kind == "norm":
            s["x"], s["residual"] = (rand(n, d) * 0.5).to(dt), h if case["residual"] else None
            s["h"] = torch.empty_like(h) if case["residual"] else None
            s["out"] = torch.empty_like(h)
            s["rstd"] = torch.empty(n, device=dev)
            s["codes"] = torch.empty(n, d, dtype=torch.float8_e4m3fn, device=dev) if case["keep"] else None
            s["scales"] = torch.empty(n, _scales(d), device=dev) if case["keep"] else None
            return s
        x = h.float()
        s["rstd"] = ((x * x).sum(1) / d + EPS).rsqrt()
        s["h"], s["codes"], s["scales"] = (None, *_encode(x)) if case["keep"] else (h, None, None)
        s["dy"] = (rand(n, d) * 0.01).to(dt)
        s["upstream"] = (rand(n, d) * 0.01).to(dt) if case["upstream"] else None
        s["y"] = torch.empty_like(h) if case["keep"] else None
        s["dx"], s["dgain"] = torch.empty_like(h), torch.empty_like(s["gain"])
        if own:
            import zero_sharded_optimizer_owned_amd as zs

            s["workspace"] = zs.rms_norm_workspace(n, d, dev)
        return s
    v = case["vocab"]
    s["weight"] = torch.empty(v, d, dtype=dt, device=dev).normal_(0, 2.0 / math.sqrt(d), generator=gen)
    s["targets"] = torch.randint(0, v, (n,), generator=gen, device=dev)
    said = s["weight"][s["targets"]].float()
    # what was said is mostly likely
    pull = (7.0 + 2.0 * rand(n, 1)) / (said * said).sum(1, keepdim=True).clamp_min(1e-2)
    s["hidden"] = (rand(n, d) + pull * said).to(dt)
    s["targets"].masked_fill_(_ignored(n).to(dev), -100)
    # answers of 1 to 64 tokens, each weighted by its length
    s["row_weight"] = 1.0 / torch.randint(1, 65, (n,), generator=gen, device=dev).float() if case["weighted"] else None
    s["divisor"] = float(max(1, n // 16))
    s["grad_scale"] = 1024.0 if case["dtype"] == "f16" else 1.0  # half precision: a loss scale
    s["stats"], s["logp"] = torch.empty(2, device=dev), torch.empty(n, device=dev)
    s["dhidden"] = torch.empty_like(s["hidden"]) if case["grad"] else None
    s["dweight"] = torch.empty_like(s["weight"]) if case["grad"] else None
    if own:
        import zero_sharded_optimizer_owned_amd as zs

        s["workspace"] = zs.linear_cross_entropy_workspace(n, v, d, grad=case["grad"], device=dev)
    return s


def _given(s, *keys):
    return {k: s[k] for k in keys if s[k] is not None}


# ---------------------------------------------------------------- the plain forms
def _plain_embed(s):
    t = s["tokens"]
    rows = s["table"][t.clamp_min(0)].float() * s["scale"]
    s["out"].copy_(torch.where((t >= 0)[:, None], rows, 0.0).to(s["out"].dtype))
    return {"out": s["out"]}


def _plain_embed_grad(s):
    t, d = s["tokens"], s["dtable"]
    wide = torch.float64 if d.dtype == torch.float32 else torch.float32  # frequent tokens: long sums
    total = torch.zeros(d.shape, dtype=wide, device=d.device)
    part = torch.where((t >= 0)[:, None], s["dout"].to(wide), 0.0)
    total.index_add_(0, t.clamp_min(0), part)
    total *= s["scale"]
    if s["case"]["accumulate"]:
        total += d
    d.copy_(total.to(d.dtype))
    return {"dtable": d}


def _plain_norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        s["h"].copy_((h + s["residual"].float()).to(s["h"].dtype))  # the norm is of what is stored
        h = s["h"].float()
    mean = (h * h).sum(1, dtype=torch.float64) / h.shape[1]
    rstd = (1 / (mean + EPS).sqrt()).float()
    s["rstd"].copy_(rstd)
    s["out"].copy_((h * rstd[:, None] * s["gain"].float()).to(s["out"].dtype))
    if s["codes"] is not None:
        codes, scales = _encode(h)
        s["codes"].copy_(codes)
        s["scales"].copy_(scales)
    return _given(s, "out", "h", "rstd", "codes", "scales")


def _plain_norm_grad(s):
    g, dy = s["gain"].float(), s["dy"].float()
    n = (s["h"].float() if s["h"] is not None else _decode(s["codes"], s["scales"])) * s["rstd"][:, None]
    if s["y"] is not None:
        s["y"].copy_((n * g).to(s["y"].dtype))
    s["dgain"].copy_((dy * n).sum(0, dtype=torch.float64).to(g.dtype).to(s["dgain"].dtype))
    dn = dy * g
    dx = (dn - n * ((dn * n).sum(1, dtype=torch.float64) / n.shape[1]).float()[:, None]) * s["rstd"][:, None]
    if s["upstream"] is not None:
        dx = dx + s["upstream"].float()
    s["dx"].copy_(dx.to(s["dx"].dtype))
    return _given(s, "dx", "dgain", "y")


def _plain_head(s):
    c, t = s["case"], s["targets"]
    h, w = s["hidden"].float(), s["weight"].float()
    x = (h @ w.t()) / c["temperature"]
    x -= x.amax(1, keepdim=True)
    counts = t >= 0
    at = torch.where(counts, t, 0)[:, None]
    said = x.gather(1, at)[:, 0].double()
    x.exp_()
    total = x.sum(1, dtype=torch.float64)
    lp = torch.where(counts, said - total.log(), 0.0)
    share = torch.where(counts, 1.0 if s["row_weight"] is None else s["row_weight"], 0.0).double() / s["divisor"]
    s["stats"].copy_(torch.stack([-(share * lp).sum(), counts.sum().double()]).float())
    s["logp"].copy_(lp.float())
    if c["grad"]:
        coef = (share * (s["grad_scale"] / c["temperature"])).float()
        x *= (coef / total).float()[:, None]
        x.scatter_add_(1, at, -coef[:, None])
        s["dhidden"].copy_((x @ w).to(s["dhidden"].dtype))
        s["dweight"].copy_((x.t() @ h).to(s["dweight"].dtype))
    return _given(s, "stats", "logp", "dhidden", "dweight")


# ---------------------------------------------------------------- the library's calls
def _own_embed(s):
    import zero_sharded_optimizer_owned_amd as zs

    zs.zero_embedding(s["table"], s["tokens"], s["out"], scale=s["scale"])
    return {"out": s["out"]}


def _own_embed_grad(s):
    import zero_sharded_optimizer_owned_amd as zs

    zs.zero_embedding_grad(s["dout"], s["tokens"], s["dtable"], scale=s["scale"], accumulate=s["case"]["accumulate"],
                           workspace=s["workspace"])
    return {"dtable": s["dtable"]}


def _own_norm(s):
    import zero_sharded_optimizer_owned_amd as zs

    zs.zero_rms_norm(s["x"], s["gain"], s["out"], residual=s["residual"], h=s["h"], eps=EPS, rstd=s["rstd"],
                     codes=s["codes"], scales=s["scales"])
    return _given(s, "out", "h", "rstd", "codes", "scales")


def _own_norm_grad(s):
    import zero_sharded_optimizer_owned_amd as zs

    if s["y"] is not None:
        zs.zero_rms_norm_restore(s["codes"], s["scales"], s["rstd"], s["gain"], s["y"])
    zs.zero_rms_norm_backward(s["dy"], s["gain"], s["rstd"], s["dx"], s["dgain"], h=s["h"], codes=s["codes"],
                              scales=s["scales"], upstream=s["upstream"], workspace=s["workspace"])
    return _given(s, "dx", "dgain", "y")


def _own_head(s):
    import zero_sharded_optimizer_owned_amd as zs

    zs.zero_linear_cross_entropy(s["hidden"], s["weight"], s["targets"], row_weight=s["row_weight"],
                                 divisor=s["divisor"], temperature=s["case"]["temperature"],
                                 grad_scale=s["grad_scale"], stats=s["stats"], logp=s["logp"], dhidden=s["dhidden"],
                                 dweight=s["dweight"], workspace=s["workspace"])
    return _given(s, "stats", "logp", "dhidden", "dweight")


PLAIN = dict(embed=_plain_embed, embed_grad=_plain_embed_grad, norm=_plain_norm, norm_grad=_plain_norm_grad,
             head=_plain_head)
OWN = dict(embed=_own_embed, embed_grad=_own_embed_grad, norm=_own_norm, norm_grad=_own_norm_grad, head=_own_head)


def run(state):
    return (OWN if own else PLAIN)[state["case"]["kind"]](state)


# ---------------------------------------------------------------- the definitions, in 64 bits
def _round_e4m3(x):
    """Nearest e4m3 value (ties to even) of numbers up to 464: 3 bits below the leading one, steps of 2^-9 below 2^-6."""
    step = torch.exp2(torch.frexp(x)[1].clamp_min(-5).double() - 4)
    return torch.round(x / step) * step


def _exact_rows(kind, s):
    case, dim = s["case"], s["case"]["dim"]
    gain = s["gain"].double()
    of = torch.arange(dim, device="cuda") // BLOCK
    if kind == "norm":
        h, out = s["x"].double(), {}
        if s["residual"] is not None:
            # the stored sum is one rounding of the exact one, and everything else starts from it
            out["h"] = h + s["residual"].double()
            h = out["h"].to(DTYPES[case["dtype"]]).double()
        out["rstd"] = (h.pow(2).mean(1) + EPS) ** -0.5
        out["out"] = torch.einsum("nd,n,d->nd", h, out["rstd"], gain)
        if case["keep"]:
            top = torch.zeros(len(h), _scales(dim), dtype=torch.float64, device="cuda")
            top.scatter_reduce_(1, of.expand(len(h), dim), h.abs(), "amax")
            top = torch.where(top < TINY_MAX, 0.0, top)
            unit = torch.where(top > 0, top / E4M3_MAX, 1.0)[:, of]
            out["codes"], out["scales"] = _round_e4m3(h / unit) * (top > 0)[:, of], top / E4M3_MAX
        return out
    r = s["rstd"].double()
    h = s["h"].double() if s["h"] is not None else s["codes"].double() * s["scales"].double()[:, of]
    n, dy = torch.einsum("nd,n->nd", h, r), s["dy"].double()
    out = {} if s["y"] is None else {"y": n * gain}
    out["dgain"] = torch.einsum("nd,nd->d", dy, n)
    along = torch.einsum("nd,nd,d->n", dy, n, gain) / dim
    out["dx"] = torch.einsum("nd,n->nd", dy * gain - n * along[:, None], r)
    if s["upstream"] is not None:
        out["dx"] += s["upstream"]
    return out


def _exact_head(case, s):
    t, n = s["targets"], case["rows"]
    live = torch.nonzero(t >= 0)[:, 0]
    h, w, said = s["hidden"][live].double(), s["weight"].double(), t[live]
    table = torch.log_softmax(torch.mm(h, w.T).div_(case["temperature"]), 1)
    lp = torch.zeros(n, dtype=torch.float64, device="cuda")
    lp[live] = table[torch.arange(len(live), device="cuda"), said]
    part = torch.full((n,), 1 / s["divisor"], dtype=torch.float64, device="cuda")
    if s["row_weight"] is not None:
        part *= s["row_weight"]
    part = part[live]
    loss = -torch.dot(part, lp[live])
    out = {"stats": torch.stack([loss, torch.tensor(float(len(live)), dtype=torch.float64, device="cuda")]), "logp": lp}
    if case["grad"]:
        slope = table.exp_()
        slope[torch.arange(len(live), device="cuda"), said] -= 1
        slope *= (part * s["grad_scale"] / case["temperature"])[:, None]
        out["dhidden"] = torch.zeros(n, case["dim"], dtype=torch.float64, device="cuda")
        out["dhidden"][live] = torch.mm(slope, w)
        out["dweight"] = torch.mm(slope.T, h)
    return out


def exact(case, seed):
    s, kind = prepare(case, seed), case["kind"]
    if kind == "head":
        out = _exact_head(case, s)
    elif kind in ("norm", "norm_grad"):
        out = _exact_rows(kind, s)
    else:
        on = torch.nonzero(s["tokens"] >= 0)[:, 0]
        if kind == "embed":
            out = {"out": torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")}
            out["out"][on] = torch.nn.functional.embedding(s["tokens"][on], s["table"]).double() * s["scale"]
        else:
            start = s["dtable"].double() if case["accumulate"] else torch.zeros(
                case["vocab"], case["dim"], dtype=torch.float64, device="cuda")
            out = {"dtable": start.index_add_(0, s["tokens"][on], s["dout"][on].double(), alpha=s["scale"])}
    # laid out as `run` lays them out
    order = dict(embed=["out"], embed_grad=["dtable"], norm=["out", "h", "rstd", "codes", "scales"],
                 norm_grad=["dx", "dgain", "y"], head=["stats", "logp", "dhidden", "dweight"])[kind]
    return {k: out[k] for k in order if k in out}
