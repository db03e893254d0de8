"""What is measured of the operators around the grouped FP8 products of a mixture
of experts: cases over their real range, the operators in their plain form, and
the calls a user makes of them.

The layout is that of the grouped products: the rows of an expert contiguous,
experts in ascending id, each one's rows filled up to a multiple of 128.  FP8 is
E4M3 with one FP32 scale per 128 columns of a row, K-block-major: s[C / 128][R].

Kinds of cases:
  route     logits -> the k experts of a token and their weights; "train" adds
            the gradient of the logits
  dispatch  the experts of all tokens -> the layout, and the tokens' activations
            in it in FP8; "train" turns them into an operand of the weight
            gradient (scales over 128 rows by 128 columns)
  combine   the experts' rows in the layout -> the weighted sum per token;
            "train" adds the gradients of the weights and of the rows (FP8),
            the latter also turned (scales over 128 rows of one column)
  swiglu    gate/up (BF16, interleaved) -> silu(gate) * up in FP8; "train" keeps
            the gate/up values in FP8 and takes the gradient from them
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
BLOCK = 128


def listed():
    return [
        # one token of a serving loop: the router of 256 experts in 8 groups, balanced by a bias
        dict(name="route 1 token of 256", kind="route", T=1, E=256, k=8, dtype="f32", scoring="sigmoid", bias=True, groups=8, top_groups=4, best=2, renorm=True, scale=2.5, mask=0.0, train=False),
        # the same router over a prompt batch
        dict(name="route 16384 tokens of 256", kind="route", T=16384, E=256, k=8, dtype="f32", scoring="sigmoid", bias=True, groups=8, top_groups=4, best=2, renorm=True, scale=2.5, mask=0.0, train=False),
        # a training step of a softmax router whose weights are not renormalised: the gradient reaches every logit
        dict(name="route train 30001 of 60", kind="route", T=30001, E=60, k=4, dtype="bf16", scoring="softmax", bias=False, groups=1, top_groups=1, best=1, renorm=False, scale=1.0, mask=0.0, train=True),
        # one token to 2 of 8 experts: latency of the layout and the quantiser
        dict(name="dispatch 1x4096 to 2 of 8", kind="dispatch", T=1, E=8, k=2, H=4096, dtype="bf16", pad=0, skip=0.0, weighted=False, train=False),
        # a prompt batch to 8 of 256 experts
        dict(name="dispatch 8192x7168 8 of 256", kind="dispatch", T=8192, E=256, k=8, H=7168, dtype="bf16", pad=0, skip=0.0, weighted=False, train=False),
        # a training step of an odd number of tokens, some experts served elsewhere, FP32 rows of a wider tensor
        dict(name="dispatch train 2001x2048 4 of 60", kind="dispatch", T=2001, E=60, k=4, H=2048, dtype="f32", pad=13, skip=0.2, weighted=False, train=True),
        # a decode batch of 64 requests
        dict(name="combine 64x4096 2 of 8", kind="combine", T=64, E=8, k=2, H=4096, weighted=True, residual=True, skip=0.0, train=False),
        # a prompt batch from 8 of 256 experts
        dict(name="combine 8192x7168 8 of 256", kind="combine", T=8192, E=256, k=8, H=7168, weighted=True, residual=False, skip=0.0, train=False),
        # a training step of a layer of 60 experts
        dict(name="combine train 4001x2048 4 of 60", kind="combine", T=4001, E=60, k=4, H=2048, weighted=True, residual=False, skip=0.1, train=True),
        # a decode batch between the products of 8 experts
        dict(name="swiglu 64x2 rows of 11008", kind="swiglu", T=64, E=8, k=2, I=11008, skip=0.0, train=False),
        # a prompt batch of 1024 tokens, each to 2 of 8 experts
        dict(name="swiglu 1024x2 rows of 11008", kind="swiglu", T=1024, E=8, k=2, I=11008, skip=0.0, train=False),
        # a training step over 8192 tokens, each to 4 of 60 small experts
        dict(name="swiglu train 8192x4 of 1408", kind="swiglu", T=8192, E=60, k=4, I=1408, skip=0.0, train=True),
    ]


def draw(rng):
    def log(lo, hi):
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return n + (n > 1 and n % 1024 == 0)

    kind = rng.choice(["route", "dispatch", "combine", "swiglu"])
    k = rng.choice([1, 2, 4, 6, 8])
    if kind == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * max(2, -(-k // groups), log(8, 512) // groups)
        need = -(-k * groups // E)  # groups that hold k experts
        train = rng.random() < 0.5
        return dict(kind=kind, T=log(1, 16384), E=E, k=k, dtype=rng.choice(["f32", "bf16"]), scoring=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, top_groups=rng.randint(need, groups), best=rng.choice([1, 2]), renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), mask=rng.choice([0.0, 0.0, 0.2]), train=train)
    E = max(k, log(4, 256))
    skip = rng.choice([0.0, 0.0, 0.2])
    if kind == "swiglu":
        I = 128 * log(1, 86)
        return dict(kind=kind, T=max(1, min(log(1, 8192), 8192 * 4 * 1408 // (k * I))), E=E, k=k, I=I, skip=skip, train=rng.random() < 0.5)
    H = 128 * log(2, 56)
    T = max(1, min(log(1, 8192), 8192 * 8 * 7168 // (k * H)))
    if kind == "dispatch":
        return dict(kind=kind, T=T, E=E, k=k, H=H, dtype=rng.choice(["bf16", "f32"]), pad=rng.choice([0, 8, 13]), skip=skip, weighted=rng.random() < 0.3, train=rng.random() < 0.5)
    weighted = rng.random() < 0.7
    return dict(kind=kind, T=T, E=E, k=k, H=H, weighted=weighted, residual=rng.random() < 0.3, skip=skip, train=weighted and rng.random() < 0.5)


def capacity(T, E, k):
    """Rows that hold the layout whatever the choice: a first row in as many
    blocks as there can be experts, then whole blocks."""
    n = T * k
    used = min(n, E)
    return BLOCK * (used + (n - used) // BLOCK)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _scale(amax):
    """amax / 448, divided: by a number torch multiplies with its reciprocal."""
    return amax / torch.full_like(amax, 448.0)


def _fp8(v):
    """v [R][C] float32 -> E4M3 values [R][C], scales [C / 128][R]."""
    R, C = v.shape
    b = v.reshape(R, C // BLOCK, BLOCK)
    s = _scale(b.abs().amax(-1))
    q = b / torch.where(s > 0, s, 1.0)[..., None]
    return q.to(FP8).reshape(R, C), s.t().contiguous()


def _fp8_values(q, s):
    R, C = q.shape
    return (q.float().reshape(R, C // BLOCK, BLOCK) * s.t()[..., None]).reshape(R, C)


def _route(l, bias, case):
    """logits [T][E] -> ids int32, scores, weights [T][k].  What decides between
    experts is held in 64 bits, the logits themselves where nothing is added."""
    E, k, G, best = case["E"], case["k"], case["groups"], case["best"]
    l = l.float()
    wide = l.double() if bias is not None or best == 2 and G > 1 else l
    s = torch.softmax(wide, 1) if case["scoring"] == "softmax" else 1.0 / (1.0 + torch.exp(-wide))
    c = s + bias.double() if bias is not None else s
    off = l == float("-inf")
    key = torch.where(off, float("-inf"), c if bias is not None else l)
    if case["top_groups"] < G:
        per = key.reshape(-1, G, E // G)
        if best == 1:
            value = per.amax(-1)
        else:
            top = torch.where(off, float("-inf"), c).reshape(-1, G, E // G).topk(2, -1).values
            value = top[..., 0] + torch.where(top[..., 1] > float("-inf"), top[..., 1], 0.0)
        keep = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        stays = torch.zeros_like(value, dtype=torch.bool).scatter(1, keep, True)
        key = torch.where(stays[..., None], per, float("-inf")).reshape(-1, E)
    v, ids = torch.sort(key, dim=1, descending=True, stable=True)  # ties: lowest index first
    none, ids = v[:, :k] == float("-inf"), ids[:, :k]
    p = torch.where(none, 0.0, s.gather(1, ids)).float()
    w = p / p.sum(1, keepdim=True).clamp_min(1e-38) if case["renorm"] else p
    return torch.where(none, -1, ids).to(torch.int32), w * case["scale"]


def _route_gradient(l, ids, g, case):
    """d sum(w g) / d l"""
    l = l.float()
    s = torch.softmax(l, 1) if case["scoring"] == "softmax" else 1.0 / (1.0 + torch.exp(-l))
    at = ids.long().clamp_min(0)
    p = torch.where(ids >= 0, s.gather(1, at), 0.0)
    g = torch.where(ids >= 0, g, 0.0) * case["scale"]
    if case["renorm"]:
        total = p.sum(1, keepdim=True).clamp_min(1e-38)
        d = (g - (g * p).sum(1, keepdim=True) / total) / total
    else:
        d = g
    d = torch.zeros_like(s).scatter_add(1, at, torch.where(ids >= 0, d, 0.0))
    if case["scoring"] == "softmax":
        return s * (d - (s * d).sum(1, keepdim=True))
    return d * s * (1.0 - s)


def _plan(ids, E, M):
    """-> rows [T][k], pairs [M], m_indices [M] int32, offsets [E + 1] int64, counts [E] int32"""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).scatter_add(0, key, torch.ones_like(key))
    padded = (counts + BLOCK - 1) // BLOCK * BLOCK
    offsets = torch.cumsum(padded, 0) - padded  # of E as well: where the layout ends
    order = torch.sort(key, stable=True).indices
    by = key[order]
    row = offsets[by] + torch.arange(n, device=ids.device) - (torch.cumsum(counts, 0) - counts)[by]
    row = torch.where(by < E, row, M)  # M: dropped
    rows = torch.empty_like(row).scatter(0, order, torch.where(by < E, row, -1))
    pairs = torch.full((M + 1,), -1, dtype=torch.int64, device=ids.device).scatter(0, row, order)[:M]
    experts = torch.where(pairs >= 0, key[pairs.clamp_min(0)], -1)
    return (rows.reshape(ids.shape).to(torch.int32), pairs.to(torch.int32), experts.to(torch.int32), offsets, counts[:E].to(torch.int32))


def _rows_of(x, pairs, k, weights):
    """The tokens' rows in the layout, zeros where there is none."""
    at = pairs.long().clamp_min(0)
    v = x.float()[at // k]
    if weights is not None:
        v = v * weights.reshape(-1)[at][:, None]
    return torch.where(pairs[:, None] >= 0, v, 0.0)


def _sum_of(c, rows, weights, residual):
    v = c.float()[rows.long().clamp_min(0)]  # [T][k][H]
    v = torch.where(rows[..., None] >= 0, v, 0.0)
    y = (v * weights[..., None] if weights is not None else v).sum(1)
    return (y + residual.float() if residual is not None else y).to(torch.bfloat16)


def _silu(g):
    sig = 1.0 / (1.0 + torch.exp(-g))
    return g * sig, sig


def _turned(q, s, across):
    """FP8 rows [R][C] -> [C][R] with scales over 128 rows by `across` columns:
    [R / 128][C / across]."""
    R, C = q.shape
    v = _fp8_values(q, s).t().reshape(C // across, across, R // BLOCK, BLOCK)
    t = _scale(v.abs().amax((1, 3)))
    v = v / torch.where(t > 0, t, 1.0)[:, None, :, None]
    return v.to(FP8).reshape(C, R), t.t().contiguous()


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _choice(g, T, E, k, skip):
    """k experts a token, some liked better than others; skip: the share of
    experts that other processes serve (their slots hold -1)."""
    liked = torch.randn(E, device="cuda", generator=g) * 0.5
    ids = (torch.randn(T, E, device="cuda", generator=g) + liked).topk(k, 1).indices.to(torch.int32)
    if skip:
        gone = torch.rand(E, device="cuda", generator=g) < skip
        ids = torch.where(gone[ids.long()], -1, ids)
    return ids


def _weights(g, ids):
    w = torch.rand(ids.shape, device="cuda", generator=g) + 0.1
    w = torch.where(ids >= 0, w, 0.0)
    return w / w.sum(1, keepdim=True).clamp_min(1e-30)


def _activations(g, rows, cols):
    """N(0, 1) with 1 % of the channels twenty times as large."""
    x = torch.randn(rows, cols, device="cuda", generator=g)
    hot = torch.randperm(cols, device="cuda", generator=g)[:cols // 100]
    x[:, hot] *= 20.0
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind, T, E, k = case["kind"], case["T"], case["E"], case["k"]

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    def zeros(*shape, dtype):
        return torch.zeros(*shape, dtype=dtype, device="cuda")

    s = dict(case=case)
    if kind == "route":
        l = randn(T, E) * 2.0
        if case["mask"]:
            l[:, torch.rand(E, device="cuda", generator=g) < case["mask"]] = float("-inf")
        s["logits"] = l.to(torch.bfloat16) if case["dtype"] == "bf16" else l
        s["bias"] = randn(E) * 0.1 if case["bias"] else None
        s["g"] = randn(T, k) * 1e-3
        s["ids"], s["weights"] = zeros(T, k, dtype=torch.int32), zeros(T, k, dtype=torch.float32)
        s["dlogits"] = torch.zeros_like(s["logits"])
        return s
    ids, M = _choice(g, T, E, k, case["skip"]), capacity(T, E, k)
    if kind == "dispatch":
        H = case["H"]
        x = _activations(g, T, H + case["pad"])[:, :H]
        s["ids"], s["x"] = ids, x.to(torch.bfloat16) if case["dtype"] == "bf16" else x
        if case["dtype"] == "bf16" and case["pad"]:  # rows of a wider tensor
            s["x"] = _activations(g, T, H + case["pad"]).to(torch.bfloat16)[:, :H]
        s["weights"] = _weights(g, ids) if case["weighted"] else None
        s["rows"], s["pairs"], s["m_indices"] = zeros(T, k, dtype=torch.int32), zeros(M, dtype=torch.int32), zeros(M, dtype=torch.int32)
        s["offsets"], s["counts"] = zeros(E + 1, dtype=torch.int64), zeros(E, dtype=torch.int32)
        s["a"], s["sa"] = zeros(M, H, dtype=torch.uint8), zeros(H // BLOCK, M, dtype=torch.float32)
        s["workspace"] = zeros(8 << 20, dtype=torch.uint8)
        if case["train"]:
            s["at"], s["sat"] = zeros(H, M, dtype=torch.uint8), zeros(M // BLOCK, H // BLOCK, dtype=torch.float32)
        return s
    s["rows"], s["pairs"], s["m_indices"], _, _ = _plan(ids, E, M)
    real = s["m_indices"][:, None] >= 0
    if kind == "combine":
        H = case["H"]
        s["c"] = torch.where(real, randn(M, H).to(torch.bfloat16), 0.0)
        s["weights"] = _weights(g, ids) if case["weighted"] else None
        s["residual"] = randn(T, H).to(torch.bfloat16) if case["residual"] else None
        s["y"] = zeros(T, H, dtype=torch.bfloat16)
        if case["train"]:
            s["dy"], s["dweights"] = (randn(T, H) * 1e-3).to(torch.bfloat16), zeros(T, k, dtype=torch.float32)
            s["dc"], s["sdc"] = zeros(M, H, dtype=torch.uint8), zeros(H // BLOCK, M, dtype=torch.float32)
            s["dct"], s["sdct"] = zeros(H, M, dtype=torch.uint8), zeros(M // BLOCK, H, dtype=torch.float32)
        return s
    I = case["I"]
    s["gu"] = torch.where(real, (randn(M, 2 * I) * 2.0).to(torch.bfloat16), 0.0)
    names = [("h", I)]
    if case["train"]:
        s["dh"] = torch.where(real, (randn(M, I) * 1e-3).to(torch.bfloat16), 0.0)
        names += [("kept", 2 * I), ("dgu", 2 * I), ("h2", I)]
    for name, C in names:
        s[name], s["s" + name] = zeros(M, C, dtype=torch.uint8), zeros(C // BLOCK, M, dtype=torch.float32)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _run_route(s):
    ids, w = _route(s["logits"], s["bias"], s["case"])
    out = dict(ids=ids, weights=w)
    if s["case"]["train"]:
        out["dlogits"] = _route_gradient(s["logits"], ids, s["g"], s["case"]).to(s["logits"].dtype)
    return out


def _run_route_own(s):
    import fp8_block_scaled_dg_amd as dg
    c = s["case"]
    dg.dg_moe_route(s["ids"], s["weights"], s["logits"], bias=s["bias"], scoring=c["scoring"], groups=c["groups"], top_groups=c["top_groups"],
                    group_best=c["best"], renormalise=c["renorm"], scale=c["scale"])
    out = dict(ids=s["ids"], weights=s["weights"])
    if c["train"]:
        dg.dg_moe_route_backward(s["dlogits"], s["g"], s["ids"], s["logits"], scoring=c["scoring"], renormalise=c["renorm"], scale=c["scale"])
        out["dlogits"] = s["dlogits"]
    return out


def _run_dispatch(s):
    case = s["case"]
    rows, pairs, m_indices, offsets, counts = _plan(s["ids"], case["E"], s["pairs"].numel())
    a, sa = _fp8(_rows_of(s["x"], pairs, case["k"], s["weights"]))
    out = dict(rows=rows, pairs=pairs, m_indices=m_indices, offsets=offsets, counts=counts, a=a, sa=sa)
    if case["train"]:
        out["at"], out["sat"] = _turned(a, sa, BLOCK)
    return out


def _run_dispatch_own(s):
    import fp8_block_scaled_dg_amd as dg
    dg.dg_moe_plan(s["rows"], s["pairs"], s["m_indices"], s["offsets"], s["counts"], s["ids"], workspace=s["workspace"])
    dg.dg_moe_dispatch_fp8(s["a"], s["sa"], s["x"], s["rows"], s["pairs"], weights=s["weights"])
    out = {**{n: s[n] for n in ("rows", "pairs", "m_indices", "offsets", "counts", "sa")}, "a": s["a"].view(FP8)}
    if s["case"]["train"]:
        dg.dg_transpose_fp8_blocks(s["at"], s["sat"], s["a"], s["sa"], block_rows=BLOCK, m_indices=s["m_indices"])
        out["at"], out["sat"] = s["at"].view(FP8), s["sat"]
    return out


def _run_combine(s):
    y = _sum_of(s["c"], s["rows"], s["weights"], s["residual"])
    if not s["case"]["train"]:
        return dict(y=y)
    rows = s["rows"]
    dot = (s["c"].float()[rows.long().clamp_min(0)] * s["dy"].float()[:, None]).sum(-1)
    dc, sdc = _fp8(_rows_of(s["dy"], s["pairs"], s["case"]["k"], s["weights"]))
    dct, sdct = _turned(dc, sdc, 1)
    return dict(y=y, dweights=torch.where(rows >= 0, dot, 0.0), dc=dc, sdc=sdc, dct=dct, sdct=sdct)


def _run_combine_own(s):
    import fp8_block_scaled_dg_amd as dg
    dg.dg_moe_combine(s["y"], s["c"], s["rows"], weights=s["weights"], residual=s["residual"])
    if not s["case"]["train"]:
        return dict(y=s["y"])
    dg.dg_moe_combine_backward(s["dc"], s["sdc"], s["dweights"], s["dy"], s["c"], s["rows"], s["pairs"], s["weights"])
    dg.dg_transpose_fp8_blocks(s["dct"], s["sdct"], s["dc"], s["sdc"], block_rows=1, m_indices=s["m_indices"])
    return dict(y=s["y"], dweights=s["dweights"], dc=s["dc"].view(FP8), sdc=s["sdc"], dct=s["dct"].view(FP8), sdct=s["sdct"])


def _run_swiglu(s):
    gu = s["gu"].float()
    M, I = gu.shape[0], gu.shape[1] // 2
    v, _ = _silu(gu[:, 0::2])
    h, sh = _fp8(v * gu[:, 1::2])
    out = dict(h=h, sh=sh)
    if s["case"]["train"]:
        kept, skept = _fp8(gu)
        gu = _fp8_values(kept, skept)
        gate, up = gu[:, 0::2], gu[:, 1::2]
        v, sig = _silu(gate)
        dh = s["dh"].float()
        dgu, sdgu = _fp8(torch.stack((dh * up * sig * (1.0 + gate * (1.0 - sig)), dh * v), -1).reshape(M, 2 * I))
        h2, sh2 = _fp8(v * up)
        out.update(kept=kept, skept=skept, dgu=dgu, sdgu=sdgu, h2=h2, sh2=sh2)
    return out


def _run_swiglu_own(s):
    import fp8_block_scaled_dg_amd as dg
    m = s["m_indices"]
    if not s["case"]["train"]:
        dg.dg_swiglu_fp8(s["h"], s["sh"], s["gu"], m_indices=m)
        return dict(h=s["h"].view(FP8), sh=s["sh"])
    dg.dg_swiglu_fp8(s["h"], s["sh"], s["gu"], s["kept"], s["skept"], m_indices=m)
    dg.dg_swiglu_fp8_backward(s["dgu"], s["sdgu"], s["dh"], s["kept"], s["skept"], s["h2"], s["sh2"], m_indices=m)
    names = ("h", "kept", "dgu", "h2")
    return {**{n: s[n].view(FP8) for n in names}, **{"s" + n: s["s" + n] for n in names}}


def run(s):
    kind = s["case"]["kind"]
    if own:
        return {"route": _run_route_own, "dispatch": _run_dispatch_own, "combine": _run_combine_own, "swiglu": _run_swiglu_own}[kind](s)
    return {"route": _run_route, "dispatch": _run_dispatch, "combine": _run_combine, "swiglu": _run_swiglu}[kind](s)


def work(case):
    """Inputs once, outputs once, without the fill up to 128 rows."""
    kind, T, E, k = case["kind"], case["T"], case["E"], case["k"]
    n = T * k * (1.0 - case.get("skip", 0.0))  # rows, in the mean
    fp8 = 1 + 4 / BLOCK
    if kind == "route":
        size = T * E * (4 if case["dtype"] == "f32" else 2)
        return {"bytes": size * (2 if case["train"] else 1) + T * k * (12 if case["train"] else 8) + 4 * E * case["bias"], "flops": T * E * (20 if case["train"] else 10)}
    if kind == "swiglu":
        I = case["I"]
        if not case["train"]:
            return {"bytes": n * I * (4 + fp8), "flops": 10 * n * I}
        # gu and dh read; h twice, kept and dgu written
        return {"bytes": n * I * (4 + 2 + 6 * fp8), "flops": 40 * n * I}
    H = case["H"]
    if kind == "dispatch":
        return {"bytes": T * H * (2 if case["dtype"] == "bf16" else 4) + n * H * fp8 + T * k * (8 + 4 * case["weighted"]) + 8 * n + case["train"] * n * H, "flops": 4 * n * H}
    moved = 2 * n * H + 2 * T * H * (1 + case["residual"]) + T * k * 8
    if case["train"]:  # dy read, the rows' gradients (both ways) and the weights' written
        moved += 2 * T * H + 2 * n * H * fp8 + 4 * T * k
    return {"bytes": moved, "flops": (6 if case["train"] else 2) * n * H}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, apart from the above
# ---------------------------------------------------------------------------

def _e4m3_64(x):
    """Every value of x (|x| <= 448) on the E4M3 grid: 3 bits after the leading
    one, steps of 2^-9 below 2^-6; halves to even."""
    step = torch.exp2((torch.frexp(x.abs().clamp_min(2.0 ** -6)).exponent - 4).double())
    return torch.round(x / step) * step


def _coded64(x, amax):
    """Codes' values of x in blocks with largest magnitudes amax, and the scales:
    as the format has it, the scale and the quotient are FP32 numbers."""
    s = (amax / torch.full_like(amax, 448.0)).float().double()
    return _e4m3_64((x / torch.where(s > 0, s, 1.0)).float().double()), s


def _blocks64(x):
    """x [R][C] float64 -> codes' values, scales [C / 128][R]"""
    q, s = torch.empty_like(x), []
    for c in range(0, x.shape[1], 128):
        part = x[:, c:c + 128]
        q[:, c:c + 128], scale = _coded64(part, part.abs().max(1, keepdim=True).values)
        s.append(scale[:, 0])
    return q, torch.stack(s)


def _times64(q, s):
    """The values that codes stand for: FP32 numbers."""
    return (q * s.t().repeat_interleave(128, 1)).float().double()


def _turned64(q, s, across):
    """codes' values [R][C] and scales -> those turned, [C][R], [R / 128][C / across]"""
    x, scales = _times64(q, s).t(), []
    q = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    for r in range(0, x.shape[1], 128):
        part = x[:, r:r + 128]
        amax = part.abs().max(1).values.view(-1, across).max(1).values
        q[:, r:r + 128], scale = _coded64(part, amax.repeat_interleave(across)[:, None])
        scales.append(scale[::across, 0])
    return q, torch.stack(scales)


def _route64(s, case):
    l = s["logits"].double()
    T, E = l.shape
    k, G = case["k"], case["groups"]
    gone = torch.isinf(l)
    score = torch.softmax(l, 1) if case["scoring"] == "softmax" else torch.sigmoid(l)
    choice = score + (s["bias"].double() if s["bias"] is not None else 0.0)
    choice = choice.masked_fill(gone, -1e30)
    if case["top_groups"] < G:
        groups = choice.view(T, G, E // G).sort(-1, descending=True).values[..., :case["best"]]
        value = groups.masked_fill((groups < -1e29) & (torch.arange(case["best"], device=l.device) > 0), 0.0).sum(-1)
        cut = torch.argsort(-value, dim=1, stable=True)[:, case["top_groups"]:]
        shut = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter(1, cut, True)
        choice = choice.masked_fill(shut.repeat_interleave(E // G, 1), -1e30)
    ids = torch.argsort(-choice, dim=1, stable=True)[:, :k]
    live = choice.gather(1, ids) > -1e29
    leaf = l.masked_fill(gone, -1e4).requires_grad_()  # e^-1e4 is 0 in 64 bits as well
    p = (torch.softmax(leaf, 1) if case["scoring"] == "softmax" else torch.sigmoid(leaf)).gather(1, ids) * live
    w = case["scale"] * (p / p.sum(1, keepdim=True).clamp_min(1e-300) if case["renorm"] else p)
    out = dict(ids=None, weights=w.detach())
    if case["train"]:
        (w * s["g"].double()).sum().backward()
        out["dlogits"] = leaf.grad
    return out


def _layout64(rows, M, values):
    """values [T k][H] at their rows"""
    out = torch.zeros(M, values.shape[1], dtype=torch.float64, device=values.device)
    at = rows.reshape(-1).long()
    out[at[at >= 0]] = values[at >= 0]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind, T, E, k = case["kind"], case["T"], case["E"], case["k"]
    if kind == "route":
        return _route64(s, case)
    if kind == "dispatch":
        M = s["pairs"].numel()
        flat, rows, at = s["ids"].reshape(-1), torch.full((T * k,), -1, dtype=torch.int64, device="cuda"), 0
        for e in range(E):
            mine = torch.nonzero(flat == e).reshape(-1)
            rows[mine] = at + torch.arange(mine.numel(), device="cuda")
            at += -(-mine.numel() // 128) * 128
        v = s["x"].double().repeat_interleave(k, 0)
        if s["weights"] is not None:
            v = (v * s["weights"].double().reshape(-1, 1)).float().double()  # an FP32 product
        a, sa = _blocks64(_layout64(rows, M, v))
        out = dict(rows=None, pairs=None, m_indices=None, offsets=None, counts=None, a=a, sa=sa)
        if case["train"]:
            out["at"], out["sat"] = _turned64(a, sa, 128)
        return out
    if kind == "combine":
        w = s["weights"].double() if s["weights"] is not None else torch.ones(T, k, dtype=torch.float64, device="cuda")
        y = s["residual"].double() if s["residual"] is not None else torch.zeros(T, case["H"], dtype=torch.float64, device="cuda")
        dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            t = torch.nonzero(s["rows"][:, j] >= 0).reshape(-1)
            c = s["c"][s["rows"][t, j].long()].double()
            y[t] = y[t] + c * w[t, j, None]
            if case["train"]:
                dw[t, j] = (c * s["dy"][t].double()).sum(1)
        if not case["train"]:
            return dict(y=y)
        v = (s["dy"].double()[:, None, :] * w[..., None]).float().double().reshape(T * k, -1)  # FP32 products
        dc, sdc = _blocks64(_layout64(s["rows"], s["pairs"].numel(), v))
        dct, sdct = _turned64(dc, sdc, 1)
        return dict(y=y, dweights=dw, dc=dc, sdc=sdc, dct=dct, sdct=sdct)
    gu = s["gu"].double()
    h, sh = _blocks64(torch.nn.functional.silu(gu[:, 0::2]) * gu[:, 1::2])
    out = dict(h=h, sh=sh)
    if case["train"]:
        kept, skept = _blocks64(gu)
        leaf = _times64(kept, skept).requires_grad_()
        v = torch.nn.functional.silu(leaf[:, 0::2]) * leaf[:, 1::2]
        v.backward(s["dh"].double())
        h2, sh2 = _blocks64(v.detach())
        dgu, sdgu = _blocks64(leaf.grad)
        out.update(kept=kept, skept=skept, dgu=dgu, sdgu=sdgu, h2=h2, sh2=sh2)
    return out
