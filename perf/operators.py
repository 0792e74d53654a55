"""What is measured of the operators that train an adapter set and serve many of them at once.

Three operators, each with a plain form (elementary torch operations in 32 bits, rounded once at
the end) and the library's call:

  multi   one shared projection for rows that belong to the requests of many adapters
          (``lora_linear_fwd_multi``);
  adamw   one AdamW step over a whole adapter set, moments in 32 bits or in blocks of 8-bit codes
          (``lora_adamw_step``; 8-bit moments are returned as the values they stand for,
          ``lora_block8_decode``);
  norm    layer norm, or the form without a mean, forward and backward with the gradients of its
          weight and bias (``lora_norm_fwd``, ``lora_norm_bwd``).

Sizes are those of the repository's workloads: the Wan2.1-1.3B q/k/v and FFN layers (1536, 4608,
8960; 32760 tokens), the 4-bit SwiGLU layer (4096, 2 x 14336), the 5120-wide sidecar layer.
"""
import math
import random
import statistics

import torch

own = False

DEV = "cuda"
BLOCK8 = 256                                   # elements per 8-bit block
LR, BETA1, BETA2, EPS, DECAY = 1e-4, 0.9, 0.999, 1e-8, 0.01


# ----------------------------------------------------------------------------------- cases
def listed():
    return [
        # one request decoding on the Wan q/k/v layer: the smallest call, latency only
        dict(name="multi decode 1 qkv", op="multi", tokens=1, inner=1536, out=4608, groups=3, rank=32, slots=8,
             base="bf16", mix="decode", bias=False),
        # a full decode batch, nearly every request with an adapter of its own
        dict(name="multi decode 64 wide", op="multi", tokens=64, inner=5120, out=5120, groups=1, rank=16, slots=64,
             base="bf16", mix="decode", bias=True),
        # the same on the 4-bit gate/up layer
        dict(name="multi decode 16 nf4", op="multi", tokens=16, inner=4096, out=28672, groups=2, rank=16, slots=16,
             base="nf4", mix="decode", bias=False),
        # a scheduler's step: ragged prompt pieces and decoding rows in one batch, an odd row count
        dict(name="multi mixed 777 up", op="multi", tokens=777, inner=1536, out=8960, groups=1, rank=64, slots=12,
             base="bf16", mix="mixed", bias=True),
        # whole prompts (a 480p latent's tokens), a few requests with long runs of rows
        dict(name="multi prompts 32760 qkv", op="multi", tokens=32760, inner=1536, out=4608, groups=3, rank=32,
             slots=8, base="bf16", mix="prompts", bias=False),
        # one layer's q/k/v adapter: six small tensors, latency
        dict(name="adamw one layer 32", op="adamw", layers=1, rank=32, width=1536, ffn=0, odd=0, state=32,
             param="master", grad="fp32"),
        # the whole model's adapters (30 layers, q/k/v and FFN), moments in 8 bits
        dict(name="adamw model 8-bit", op="adamw", layers=30, rank=64, width=1536, ffn=8960, odd=5, state=8,
             param="master", grad="fp32"),
        # the same with moments in 32 bits and fp32 adapters
        dict(name="adamw model 32-bit", op="adamw", layers=30, rank=64, width=1536, ffn=8960, odd=5, state=32,
             param="fp32", grad="fp32"),
        # the norm ahead of a decode batch's projection
        dict(name="norm fwd 16 rows", op="norm", dir="fwd", rows=16, cols=5120, kind="rms", affine=True, dtype="bf16"),
        # a prompt's norm, forward
        dict(name="norm fwd 32760", op="norm", dir="fwd", rows=32760, cols=1536, kind="layer", affine=True,
             dtype="bf16"),
        # and backward, with the weight's and bias's gradients
        dict(name="norm bwd 32760", op="norm", dir="bwd", rows=32760, cols=1536, kind="layer", affine=True,
             dtype="bf16"),
        # an odd width in fp32
        dict(name="norm bwd odd fp32", op="norm", dir="bwd", rows=1111, cols=4099, kind="layer", affine=True,
             dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["multi", "multi", "adamw", "norm"])
    if op == "multi":
        base = rng.choice(["bf16", "bf16", "nf4"])
        step = 64 if base == "nf4" else 8
        inner = max(step, _log(rng, 256, 14336) // step * step)
        groups = rng.choice([1, 1, 2, 3])
        out_g = max(64, _log(rng, 256, 14336 // groups) // 8 * 8)
        rank = rng.choice([8, 16, 24, 32, 64, 128])
        tokens = _log(rng, 1, 32760)
        tokens = min(tokens, max(1, 231_000_000_000 // (inner * out_g * groups)))
        slots = _log(rng, 1, 64)
        slots = min(slots, max(1, 8192 // (groups * rank)))      # the plain form multiplies by every slot
        mix = rng.choice(["decode", "mixed", "prompts"])
        if tokens > 2048 and mix == "decode":
            mix = "prompts"
        return dict(op="multi", tokens=tokens, inner=inner, out=out_g * groups, groups=groups, rank=rank, slots=slots,
                    base=base, mix=mix, bias=rng.random() < 0.5)
    if op == "adamw":
        width, rank = _log(rng, 256, 5120), rng.choice([4, 8, 16, 32, 64])
        ffn = rng.choice([0, _log(rng, 512, 14336)])
        per = rank * (6 * width + 2 * (width + ffn) * (1 if ffn else 0))
        layers = max(1, min(_log(rng, 1, 40), 49_000_000 // per))
        return dict(op="adamw", layers=layers, rank=rank, width=width, ffn=ffn, odd=rng.randrange(0, 12),
                    state=rng.choice([8, 32]), param=rng.choice(["master", "fp32", "bf16"]),
                    grad=rng.choice(["fp32", "fp32", "bf16"]))
    rows, cols = _log(rng, 1, 32760), _log(rng, 64, 14336)
    rows = min(rows, max(1, 50_000_000 // cols))
    return dict(op="norm", dir=rng.choice(["fwd", "bwd"]), rows=rows, cols=cols, kind=rng.choice(["layer", "rms"]),
                affine=rng.random() < 0.8, dtype=rng.choice(["bf16", "bf16", "fp32"]))


# ---------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 13)
    return g


def _normal(g, shape, std, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _runs(r, total, count):
    """`count` positive lengths that add up to `total`."""
    count = max(1, min(count, total))
    cuts = sorted(r.sample(range(1, total), count - 1)) if count > 1 else []
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _slots_of_rows(case, seed):
    """The slot of each row: requests of one row each (decode), long runs (prompts), or both.
    About one request in ten uses no adapter (-1)."""
    r = random.Random(int(seed) * 31 + 7)
    tokens, slots = case["tokens"], case["slots"]
    pick = lambda: -1 if r.random() < 0.1 else r.randrange(slots)  # noqa: E731
    if case["mix"] == "decode":
        return [pick() for _ in range(tokens)]
    single = min(tokens // 3, 100) if case["mix"] == "mixed" else 0
    rows = []
    for n in _runs(r, tokens - single, max(1, min(2 * slots, 1 + (tokens - single) // 40))):
        rows += [pick()] * n
    return rows + [pick() for _ in range(single)]


def _multi_inputs(case, seed):
    g = _gen(seed)
    t, k, n, gr, rk, sl = (case[x] for x in ("tokens", "inner", "out", "groups", "rank", "slots"))
    s = {"x": _normal(g, (t, k), 1.0)}
    if case["base"] == "nf4":
        s["codes"] = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
        s["absmax"] = (torch.randn((n * k // 64,), generator=g, device=DEV).abs() + 0.1) * (2.0 / math.sqrt(k))
    else:
        s["w"] = _normal(g, (n, k), 1.0 / math.sqrt(k))
    s["bias"] = _normal(g, (n,), 0.1) if case["bias"] else None
    s["a"] = _normal(g, (sl, gr * rk, k), 1.0 / math.sqrt(k))
    s["b"] = _normal(g, (sl, n, rk), 0.02)
    s["scale"] = torch.rand((sl,), generator=g, device=DEV) + 0.5
    s["slot"] = torch.tensor(_slots_of_rows(case, seed), dtype=torch.int32, device=DEV)
    s["row_scale"] = torch.rand((t,), generator=g, device=DEV) * 0.5 + 0.75
    return s


def _adamw_sizes(case):
    """Element counts of the set's tensors: per layer q/k/v factors A [rank, width], B [width, rank], and
    with an FFN the up and down factors; `odd` norm and bias vectors with odd lengths."""
    rk, w, f = case["rank"], case["width"], case["ffn"]
    sizes = []
    for _ in range(case["layers"]):
        sizes += [rk * w] * 6
        if f:
            sizes += [rk * w, f * rk, rk * f, w * rk]
    return sizes + [w - 1 - 2 * i for i in range(case["odd"])]


def _adamw_inputs(case, seed):
    g = _gen(seed)
    sizes = _adamw_sizes(case)
    # every tensor is a view of one buffer, starting at a multiple of the 8-bit block, so that the
    # buffers can be compared whole; the gaps hold zeros and stay so
    starts, n = [], 0
    for z in sizes:
        starts.append(n)
        n += -(-z // BLOCK8) * BLOCK8
    spans = [(b, b + z) for b, z in zip(starts, sizes)]
    edge = torch.zeros(n + 1, device=DEV, dtype=torch.int32)
    edge.index_add_(0, torch.tensor([b for b, _ in spans], device=DEV), torch.ones(len(spans), device=DEV, dtype=torch.int32))
    edge.index_add_(0, torch.tensor([e for _, e in spans], device=DEV), -torch.ones(len(spans), device=DEV, dtype=torch.int32))
    used = edge.cumsum(0)[:n].float()
    rand = lambda std: torch.randn((n,), generator=g, device=DEV) * used * std  # noqa: E731
    s = {"n": n, "spans": spans, "step": 100, "case": case}
    p = rand(0.02)
    if case["param"] == "fp32":
        s["p"], s["master"] = p, None
    else:
        s["p"] = p.to(torch.bfloat16)
        s["master"] = p if case["param"] == "master" else None
    # gradients whose size differs from element to element, as trained factors' do
    size = torch.exp(torch.randn((n,), generator=g, device=DEV) * 1.5 - 6.0)
    s["grad"] = (rand(1.0) * size).to(torch.float32 if case["grad"] == "fp32" else torch.bfloat16)
    m = rand(0.3) * size
    v = (torch.rand((n,), generator=g, device=DEV) + 0.2) * size * size * used
    del size
    if case["state"] == 8:
        s["mq"], s["ms"] = _encode(m, True)
        s["vq"], s["vs"] = _encode(v, False)
    else:
        s["m"], s["v"] = m, v
    return s


def _norm_inputs(case, seed):
    g = _gen(seed)
    t, c = case["rows"], case["cols"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    rows = torch.rand((t, 1), generator=g, device=DEV)
    x = (torch.randn((t, c), generator=g, device=DEV) * (0.5 + rows) + (rows * 2 - 0.5)).to(dt)
    s = {"x": x, "kind": case["kind"], "dir": case["dir"], "w": None, "b": None}
    if case["affine"]:
        s["w"] = (1 + torch.randn((c,), generator=g, device=DEV) * 0.1).to(dt)
        if case["kind"] == "layer":
            s["b"] = (torch.randn((c,), generator=g, device=DEV) * 0.1).to(dt)
    if case["dir"] == "bwd":
        s["dy"] = torch.randn((t, c), generator=g, device=DEV).to(dt)
        f = x.float()
        mean = f.mean(1) if case["kind"] == "layer" else torch.zeros((t,), device=DEV)
        var = (f - mean[:, None]).square().mean(1)
        s["stats"] = torch.stack([mean, 1 / torch.sqrt(var + 1e-5)])     # what the forward saved
    return s


def prepare(case, seed):
    s = {"multi": _multi_inputs, "adamw": _adamw_inputs, "norm": _norm_inputs}[case["op"]](case, seed)
    s["op"] = case["op"]
    if own:
        _handles(s, case)
    return s


def _handles(s, case):
    """What a program of the library's user keeps between calls: the bank and workspace of a layer,
    the plan of an adapter set, the views of its tensors."""
    import weight_patches_gb300 as wpg
    if case["op"] == "multi":
        s["bank"] = wpg.AdapterBank(s["a"], s["b"], s["scale"], case["groups"])
        s["weight"] = wpg.NF4Weight(s["codes"], s["absmax"], case["out"], case["inner"]) if "codes" in s else s["w"]
        need = wpg.lora_multi_workspace_size(s["x"], s["weight"], s["bank"])
        s["workspace"] = torch.empty(max(need, 1), dtype=torch.uint8, device=DEV)
    elif case["op"] == "adamw":
        cut = lambda t: None if t is None else [t[a:b] for a, b in s["spans"]]  # noqa: E731
        if case["state"] == 8:
            blocks = [(a // BLOCK8, -(-b // BLOCK8)) for a, b in s["spans"]]
            m = [wpg.Block8(s["mq"][a:b], s["ms"][i:j]) for (a, b), (i, j) in zip(s["spans"], blocks)]
            v = [wpg.Block8(s["vq"][a:b], s["vs"][i:j]) for (a, b), (i, j) in zip(s["spans"], blocks)]
        else:
            m, v = cut(s["m"]), cut(s["v"])
        s["plan"] = wpg.lora_adamw_plan(cut(s["p"]), m, v, masters=cut(s["master"]))
        s["grads"] = cut(s["grad"])
    elif case["dir"] == "bwd":
        need = wpg.lora_norm_bwd_workspace_size(s["x"])
        s["workspace"] = torch.empty(max(need, 1), dtype=torch.uint8, device=DEV)


# ------------------------------------------------------------------------------------ runs
def run(state):
    return {"multi": _run_multi, "adamw": _run_adamw, "norm": _run_norm}[state["op"]](state)


def _levels():
    """The 16 NormalFloat levels: normal quantiles evenly spaced in probability on each side of an
    exact zero, scaled to [-1, 1]."""
    top = 0.5 * ((1 - 1 / 30) + (1 - 1 / 32))
    q = torch.special.ndtri(torch.linspace(top, 0.5, 9, dtype=torch.float64)[:-1])
    r = -torch.special.ndtri(torch.linspace(top, 0.5, 8, dtype=torch.float64)[:-1])
    v = torch.cat([r, torch.zeros(1, dtype=torch.float64), q.flip(0)])
    return (v / v.abs().max()).to(torch.float32)


_LEVELS = None


def _weight(s):
    """W in 32 bits; a 4-bit one as the bf16 values its codes stand for."""
    global _LEVELS
    if "w" in s:
        return s["w"].float()
    if _LEVELS is None:
        _LEVELS = _levels().to(DEV)
    c = s["codes"]
    codes = torch.stack([c >> 4, c & 15], dim=-1).reshape(-1, 64)
    return (_LEVELS[codes.int()] * s["absmax"][:, None]).to(torch.bfloat16).float().view(c.shape[0], -1)


def _run_multi(s):
    if own:
        import weight_patches_gb300 as wpg
        return wpg.lora_linear_fwd_multi(s["x"], s["weight"], s["bias"], s["bank"], s["slot"],
                                         row_scale=s["row_scale"], workspace=s["workspace"])
    x, a, b, slot = s["x"].float(), s["a"].float(), s["b"].float(), s["slot"]
    t, (sl, n, rk) = x.shape[0], b.shape
    gr = a.shape[1] // rk
    y = x @ _weight(s).t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    h = (x @ a.reshape(sl * gr * rk, -1).t()).view(t, sl, gr, rk)
    scale = s["scale"][slot.clamp(min=0).long()] * s["row_scale"]
    mine = slot[:, None] == torch.arange(sl, device=DEV, dtype=torch.int32)
    h = torch.where(mine[:, :, None, None], h * scale[:, None, None, None], 0.0)
    h = h.permute(2, 0, 1, 3).reshape(gr, t, sl * rk)
    b = b.view(sl, gr, n // gr, rk).permute(1, 0, 3, 2).reshape(gr, sl * rk, n // gr)
    return (y + (h @ b).permute(1, 0, 2).reshape(t, n)).to(torch.bfloat16)


def _encode(x, signed):
    """Blocks of 256 values as 8-bit codes and one scale each: the square (signed) or the fourth power
    (unsigned, a value above zero never coded as zero) of the code's share of the largest code."""
    b = x.view(-1, BLOCK8)
    top = b.abs().amax(1)
    share = torch.where(top[:, None] > 0, b.abs() / top[:, None], 0.0)
    if signed:
        q = torch.round(127 * torch.sqrt(share))
        q = torch.where(b < 0, -q, q).to(torch.int8)
    else:
        q = torch.round(255 * torch.sqrt(torch.sqrt(share)))
        q = torch.where(b > 0, q.clamp(min=1), q).to(torch.uint8)
    return q.view(-1), top


def _decode(q, top, signed):
    u = q.view(-1, BLOCK8).float() / (127 if signed else 255)
    u = u * u.abs() if signed else (u * u) * (u * u)
    return (u * top[:, None]).view(-1)


def _run_adamw(s):
    s["step"] += 1
    eight = s["case"]["state"] == 8
    if own:
        import weight_patches_gb300 as wpg
        wpg.lora_adamw_step(s["plan"], s["grads"], lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY,
                            step=s["step"], grad_scale=0.5)
        if eight:
            m, v = wpg.lora_block8_decode(s["mq"], s["ms"]), wpg.lora_block8_decode(s["vq"], s["vs"])
        else:
            m, v = s["m"], s["v"]
        return {"p": s["p"], "master": s["master"], "m": m, "v": v}
    f = lambda x: torch.tensor(x, dtype=torch.float32).item()  # noqa: E731
    m = _decode(s["mq"], s["ms"], True) if eight else s["m"]
    v = _decode(s["vq"], s["vs"], False) if eight else s["v"]
    g = s["grad"].float() * 0.5
    m = f(BETA1) * m + f(1 - BETA1) * g
    v = f(BETA2) * v + f(1 - BETA2) * (g * g)
    den = torch.sqrt(v) * f(1 / math.sqrt(1 - BETA2 ** s["step"])) + f(EPS)
    p = s["master"] if s["master"] is not None else s["p"].float()
    p = p * f(1 - LR * DECAY) - f(LR / (1 - BETA1 ** s["step"])) * (m / den)
    if s["master"] is not None:
        s["master"] = p
    s["p"] = p.to(s["p"].dtype)
    if eight:
        s["mq"], s["ms"] = _encode(m, True)
        s["vq"], s["vs"] = _encode(v, False)
        m, v = _decode(s["mq"], s["ms"], True), _decode(s["vq"], s["vs"], False)
    else:
        s["m"], s["v"] = m, v
    return {"p": s["p"], "master": s["master"], "m": m, "v": v}


def _run_norm(s):
    layer = s["kind"] == "layer"
    if own:
        import weight_patches_gb300 as wpg
        kind = wpg.WP_NORM_LAYER if layer else wpg.WP_NORM_RMS
        if s["dir"] == "fwd":
            y, stats = wpg.lora_norm_fwd(s["x"], s["w"], s["b"], eps=1e-5, kind=kind)
            return {"y": y, "mean": stats[0] if layer else None, "rstd": stats[1]}
        dx, dw, db = wpg.lora_norm_bwd(s["dy"], s["x"], s["w"], s["stats"], kind=kind, workspace=s["workspace"],
                                       need_db=layer)
        return {"dx": dx, "dw": dw, "db": db}
    x = s["x"].float()
    w = s["w"].float() if s["w"] is not None else None
    if s["dir"] == "fwd":
        mean = x.mean(1) if layer else None
        c = x - mean[:, None] if layer else x
        rstd = 1 / torch.sqrt((c * c).mean(1) + 1e-5)
        y = c * rstd[:, None]
        if w is not None:
            y = y * w
        if s["b"] is not None:
            y = y + s["b"].float()
        return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}
    dy = s["dy"].float()
    mean, rstd = s["stats"][0], s["stats"][1]
    xh = ((x - mean[:, None]) if layer else x) * rstd[:, None]
    h = dy * w if w is not None else dy
    dx = h - xh * (h * xh).mean(1, keepdim=True)
    if layer:
        dx = dx - h.mean(1, keepdim=True)
    dx = dx * rstd[:, None]
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * xh).sum(0), "db": dy.sum(0) if layer else None}


# ------------------------------------------------------------------------------------ work
def work(case):
    if case["op"] == "multi":
        t, k, n, gr, rk, sl = (case[x] for x in ("tokens", "inner", "out", "groups", "rank", "slots"))
        # the expected number of different slots among the requests
        r = t if case["mix"] == "decode" else min(t, 2 * sl + (min(t // 3, 100) if case["mix"] == "mixed" else 0))
        present = sl * (1 - (1 - 0.9 / sl) ** r)
        weight = n * k * (2 if case["base"] == "bf16" else 0.5 + 4 / 64)
        return {"bytes": weight + 2 * t * (k + n) + 2 * present * rk * (gr * k + n) + 8 * t,
                "flops": 2 * t * (k * n + 0.9 * rk * (gr * k + n))}
    if case["op"] == "adamw":
        n = sum(_adamw_sizes(case))
        each = {"master": 10, "fp32": 8, "bf16": 4}[case["param"]] + (4 if case["grad"] == "fp32" else 2)
        # 8 bits: codes and scales read and written, and the 32-bit values returned
        each += 16 if case["state"] == 32 else 4 + 16 / BLOCK8 + 8
        return {"bytes": n * each, "flops": n * 16}
    n = case["rows"] * case["cols"]
    size = 2 if case["dtype"] == "bf16" else 4
    if case["dir"] == "fwd":
        return {"bytes": 2 * n * size + 2 * case["cols"] * size + 8 * case["rows"], "flops": 8 * n}
    return {"bytes": 3 * n * size + case["cols"] * (size + 8) + 8 * case["rows"], "flops": 14 * n}


# ------------------------------------------------------------------------- 64-bit definition
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "multi":
        return _exact_multi(case, s)
    if case["op"] == "adamw":
        return _exact_adamw(case, s)
    return _exact_norm(case, s)


def _exact_weight(case, s):
    if case["base"] == "bf16":
        return s["w"].double()
    inv = statistics.NormalDist().inv_cdf
    top = ((1 - 1 / 30) + (1 - 1 / 32)) / 2
    pos = [inv(top + (0.5 - top) * i / 8) for i in range(8)]
    neg = [-inv(top + (0.5 - top) * i / 7) for i in range(7)]
    lev = torch.tensor(sorted(neg + [0.0] + pos), dtype=torch.float64)
    lev = (lev / lev.abs().max()).float().to(DEV)          # the codebook is held in 32 bits
    n, k = case["out"], case["inner"]
    q = torch.empty((n, k), dtype=torch.long, device=DEV)
    q[:, 0::2] = s["codes"].long() // 16
    q[:, 1::2] = s["codes"].long() % 16
    # a 4-bit weight is by definition the bf16 rounding of the 32-bit product
    scale = s["absmax"].view(n, k // 64).repeat_interleave(64, dim=1)
    return (lev[q] * scale).bfloat16().double()


def _exact_multi(case, s):
    w = _exact_weight(case, s)
    x = s["x"].double()
    y = torch.matmul(x, w.T)
    if s["bias"] is not None:
        y += s["bias"].double()
    rk, gr = case["rank"], case["groups"]
    og = case["out"] // gr
    for a in range(case["slots"]):
        rows = torch.nonzero(s["slot"] == a).flatten()
        if rows.numel() == 0:
            continue
        st = s["scale"][a].double() * s["row_scale"][rows].double()
        for g in range(gr):
            h = torch.matmul(x[rows], s["a"][a, g * rk:(g + 1) * rk].double().T) * st[:, None]
            cols = slice(g * og, (g + 1) * og)
            y[rows, cols] = y[rows, cols] + torch.matmul(h, s["b"][a, cols].double().T)
    return y


def _exact_block8(values, signed):
    """The 8-bit values that 64-bit values are held as: nearest in the root's domain."""
    out = values.clone().view(-1, BLOCK8)
    top = out.abs().max(dim=1, keepdim=True).values
    share = out.abs() / torch.where(top == 0, torch.ones_like(top), top)
    if signed:
        return (out.sign() * (share.pow(0.5) * 127).round().div(127).pow(2) * top).view(-1)
    code = (share.pow(0.25) * 255).round()
    code = torch.maximum(code, (out > 0).double())
    return (code.div(255).pow(4) * top).view(-1)


def _exact_adamw(case, s):
    t = s["step"] + 1
    g = s["grad"].double() * 0.5
    if case["state"] == 8:
        um, uv = s["mq"].double().view(-1, BLOCK8) / 127, s["vq"].double().view(-1, BLOCK8) / 255
        m0 = (um.sign() * um.square() * s["ms"].double()[:, None]).reshape(-1)
        v0 = (uv ** 4 * s["vs"].double()[:, None]).reshape(-1)
    else:
        m0, v0 = s["m"].double(), s["v"].double()
    m = BETA1 * m0 + (1 - BETA1) * g
    v = BETA2 * v0 + (1 - BETA2) * g.square()
    p = (s["master"] if s["master"] is not None else s["p"]).double()
    p = p - LR * DECAY * p - LR * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
    if case["state"] == 8:
        m, v = _exact_block8(m, True), _exact_block8(v, False)
    return {"p": p, "master": p if s["master"] is not None else None, "m": m, "v": v}


def _exact_norm(case, s):
    x = s["x"].double()
    c = x.shape[1]
    if case["dir"] == "fwd":
        mu = x.sum(1, keepdim=True) / c if case["kind"] == "layer" else torch.zeros_like(x[:, :1])
        r = torch.rsqrt((x - mu).pow(2).sum(1, keepdim=True) / c + 1e-5)
        y = (x - mu) * r
        if s["w"] is not None:
            y = y * s["w"].double()
        if s["b"] is not None:
            y = y + s["b"].double()
        return {"y": y, "mean": mu[:, 0] if case["kind"] == "layer" else None, "rstd": r[:, 0]}
    mu, r = s["stats"][0].double()[:, None], s["stats"][1].double()[:, None]
    z = (x - mu) * r
    dy = s["dy"].double()
    h = dy if s["w"] is None else dy * s["w"].double()
    dot = (h * z).sum(1, keepdim=True) / c
    avg = h.sum(1, keepdim=True) / c if case["kind"] == "layer" else 0.0
    return {"dx": r * (h - avg - z * dot), "dw": torch.einsum("tc,tc->c", dy, z),
            "db": dy.sum(0) if case["kind"] == "layer" else None}
