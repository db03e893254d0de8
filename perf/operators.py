"""What is measured of the 4-bit (MXFP4) operators and of the mixture-of-experts
layer for a few tokens: cases over their real range, the operators in their
plain form, and the calls a user makes of them.

MXFP4: E2M1 codes (0 .5 1 1.5 2 3 4 6; bit 3 is the sign), element k of a row
in nibble k % 2 of byte k // 2, and one E8M0 exponent byte per 32 elements of
a row, four in an int32, K-block-major: sf[ceil(K / 128)][rows].

Kinds of cases:
  quantise  x -> codes and scales, and back to the values they stand for
            (rowwise, transposed or both, from one x)
  product   C = A . B^T, both MXFP4 (training and prompt shapes, decode)
  a16       C = A . B^T with BF16 A that is not quantised (single tokens up)
  linear    a linear layer's forward and backward: y, dx, dw from BF16 x, w
            and dy, every product in MXFP4
  moe       router logits -> top-k -> experts (gate/up, SwiGLU, down) ->
            weighted sum, expert weights in FP8 blocks or MXFP4
"""
import math

import torch

own = False

#: a split-K workspace as a serving process keeps it: zero-filled once
WORKSPACE = 32 << 20


def listed():
    return [
        # decode activations of a 64-request batch: latency of the quantiser
        dict(name="quantise 64x4096 bf16", kind="quantise", rows=64, cols=4096, dtype="bf16", way="row", pad=0),
        # a weight quantised once per step for the forward and the input gradient
        dict(name="quantise 8192x8192 both", kind="quantise", rows=8192, cols=8192, dtype="bf16", way="both", pad=0),
        # prompt-sized projection of the dense workload
        dict(name="product 4096x7168x2048", kind="product", M=4096, N=7168, K=2048),
        # the dense workload's square
        dict(name="product 8192x8192x8192", kind="product", M=8192, N=8192, K=8192),
        # a decode batch on the dense workload's down projection
        dict(name="product 64x7168x16384", kind="product", M=64, N=7168, K=16384),
        # one token through a wide projection, activations left in BF16
        dict(name="a16 1x24576x1536", kind="a16", M=1, N=24576, K=1536),
        # a decode batch, odd number of requests
        dict(name="a16 33x7168x16384", kind="a16", M=33, N=7168, K=16384),
        # a training step of one layer over an odd number of tokens
        dict(name="linear 2001x4096x4096", kind="linear", M=2001, N=4096, K=4096),
        dict(name="linear 300x1000x2080", kind="linear", M=300, N=1000, K=2080),
        # one token through the decode workload's layer
        dict(name="moe 1 token fp8 8x4096x11008", kind="moe", T=1, E=8, k=2, H=4096, I=11008, fmt="fp8", mask=0.0, scoring="softmax"),
        # its batch of 64 requests, experts in 4 bits
        dict(name="moe 64 tokens mxfp4 8x4096x11008", kind="moe", T=64, E=8, k=2, H=4096, I=11008, fmt="mxfp4", mask=0.0, scoring="softmax"),
        # many small experts, an odd number of tokens, some experts switched off
        dict(name="moe 13 tokens fp8 60x2048x1408", kind="moe", T=13, E=60, k=4, H=2048, I=1408, fmt="fp8", mask=0.1, scoring="sigmoid"),
    ]


def draw(rng):
    def log(lo, hi):  # the round sizes are the listed cases'
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return n + (n % 1024 == 0)

    def mult(m, lo, hi):  # odd multiples: they end inside every larger tile
        return m * (log(lo / m, hi / m) | 1)

    kind = rng.choice(["quantise", "product", "product", "a16", "linear", "moe", "moe"])
    if kind == "quantise":
        return dict(kind=kind, rows=log(1, 8192), cols=log(32, 8192), dtype=rng.choice(["bf16", "f32"]), way=rng.choice(["row", "transposed", "both"]), pad=rng.choice([0, 8, 13]))
    if kind == "product":
        if rng.random() < 0.4:
            return dict(kind=kind, M=log(1, 64), N=log(128, 24576), K=mult(32, 128, 16384))
        return dict(kind=kind, M=log(65, 8192), N=log(128, 8192), K=mult(32, 128, 8192))
    if kind == "a16":
        return dict(kind=kind, M=log(1, 64), N=log(128, 24576), K=mult(32, 128, 16384))
    if kind == "linear":
        return dict(kind=kind, M=log(16, 4096), N=log(128, 4096), K=mult(32, 128, 4096))
    fmt = rng.choice(["fp8", "mxfp4"])
    m = 128 if fmt == "fp8" else 32
    E = log(4, 256)
    H, most = mult(m, 256, 4096), 8 * 4096 * 11008
    I = mult(m, 128, min(11008, max(256, most // (E * H))))
    while E * H * I > most and I > m:
        I = max(m, I // 2 // m * m)
    return dict(kind=kind, T=log(1, 64), E=E, k=min(E, rng.choice([1, 2, 4, 6, 8])), H=H, I=I, fmt=fmt, mask=rng.choice([0.0, 0.0, 0.3]), scoring=rng.choice(["softmax", "sigmoid"]))


# ---------------------------------------------------------------------------
# the formats in plain form (32 bits)
# ---------------------------------------------------------------------------

def _grid(like):
    return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=like.device)


def _quantise(x):
    """x [R][C] -> codes uint8 [R][C32 / 2], sf int32 [ceil(C / 128)][R];
    C32 = C rounded up to 32, filled with zeros."""
    R, C = x.shape
    C32 = -(-C // 32) * 32
    v = torch.nn.functional.pad(x.float(), (0, C32 - C)).reshape(R, C32 // 32, 32)
    field = v.abs().amax(-1).view(torch.int32) >> 23
    e = torch.where(field == 255, field, (field - 2).clamp_min(0))
    v = torch.ldexp(v, (127 - e).clamp_min(-126)[..., None])
    a = v.abs()
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code += torch.signbit(v).to(torch.uint8) * 8
    code = code.reshape(R, C32 // 2, 2)
    q = code[..., 0] | (code[..., 1] << 4)
    words = -(-C // 128)
    e = torch.nn.functional.pad(e.to(torch.uint8), (0, 4 * words - e.shape[1]))
    sf = e.reshape(R, words, 4).view(torch.int32).reshape(R, words).t().contiguous()
    return q, sf


def _exponents(sf, blocks):
    """sf [..][words][rows] int32 -> exponent bytes [..][rows][blocks]."""
    e = sf.transpose(-1, -2).contiguous().view(torch.uint8)
    return e[..., :blocks].int()


def _dequantise(q, sf):
    """-> float32 [..][rows][2 * bytes]"""
    C32 = 2 * q.shape[-1]
    g = _grid(q)
    pair = torch.stack((g[torch.arange(256, device=q.device) % 16], g[torch.arange(256, device=q.device) // 16]), -1)
    v = pair[q.int()].reshape(*q.shape[:-1], C32 // 32, 32)
    e = _exponents(sf, C32 // 32)
    s = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e - 127)
    s = torch.where(e == 255, float("nan"), s)
    return (v * s[..., None]).reshape(*q.shape[:-1], C32)


def _fp8_values(codes, s):
    """codes [E][N][K] E4M3, s [E][K / 128][ceil(N / 128)] -> float32."""
    E, N, K = codes.shape
    v = codes.view(torch.float8_e4m3fn).float().reshape(E, N, K // 128, 128)
    per_row = s.transpose(1, 2).repeat_interleave(128, 1)[:, :N]
    return (v * per_row[..., None]).reshape(E, N, K)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _quantise_fp8(w):
    """w [N][K] (K % 128 == 0) -> E4M3 codes, scales [K / 128][ceil(N / 128)]."""
    N, K = w.shape
    n = -(-N // 128) * 128
    b = torch.nn.functional.pad(w, (0, 0, 0, n - N)).reshape(n // 128, 128, K // 128, 128)
    s = b.abs().amax((1, 3)) / 448.0
    q = (b / s.clamp_min(1e-30)[:, None, :, None]).reshape(n, K)[:N]
    return q.to(torch.float8_e4m3fn).view(torch.uint8), s.t().contiguous()


def _activations(g, rows, cols):
    """N(0, 1) with 1 % of the channels twenty times as large."""
    x = torch.randn(rows, cols, device="cuda", generator=g)
    hot = torch.randperm(cols, device="cuda", generator=g)[:cols // 100]
    x[:, hot] *= 20.0
    return x


def _experts(g, E, N, K, fmt):
    parts = [(_quantise_fp8 if fmt == "fp8" else _quantise)(torch.randn(N, K, device="cuda", generator=g) * 0.02) for _ in range(E)]
    return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind = case["kind"]
    bf16 = dict(device="cuda", dtype=torch.bfloat16)
    s = dict(case=case)
    if kind == "quantise":
        x = _activations(g, case["rows"], case["cols"] + case["pad"])
        x = x.to(torch.bfloat16) if case["dtype"] == "bf16" else x
        s["x"] = x[:, :case["cols"]]  # a slice of a wider tensor where pad is not 0
    elif kind in ("product", "a16"):
        M, N, K = case["M"], case["N"], case["K"]
        a = _activations(g, M, K)
        s["a"], s["sa"] = _quantise(a) if kind == "product" else (a.to(torch.bfloat16), None)
        s["b"], s["sb"] = _quantise(torch.randn(N, K, device="cuda", generator=g) * 0.02)
        s["c"] = torch.empty(M, N, **bf16)
        s["workspace"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device="cuda")
    elif kind == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = _activations(g, M, K).to(torch.bfloat16)
        s["w"] = (torch.randn(N, K, device="cuda", generator=g) * 0.02).to(torch.bfloat16)
        s["dy"] = (torch.randn(M, N, device="cuda", generator=g) * 1e-3).to(torch.bfloat16)
        s["workspace"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device="cuda")
    else:
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        s["x"] = _activations(g, T, H).to(torch.bfloat16)
        s["logits"] = torch.randn(T, E, device="cuda", generator=g) * 2.0
        if case["mask"]:  # experts that this process does not serve
            s["logits"][:, torch.rand(E, device="cuda", generator=g) < case["mask"]] = float("-inf")
        s["w13"], s["s13"] = _experts(g, E, 2 * I, H, case["fmt"])  # row 2i gate, 2i + 1 up
        s["w2"], s["s2"] = _experts(g, E, H, I, case["fmt"])
        s["y"] = torch.empty(T, H, **bf16)
        s["ids"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty(T, k, device="cuda")
        # the SwiGLU outputs of every (token, slot)
        s["workspace"] = torch.zeros(max(WORKSPACE, 4 * T * k * I), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _run_quantise(s):
    x, way, dtype = s["x"], s["case"]["way"], s["x"].dtype
    ways = [x] * (way != "transposed") + [x.t()] * (way != "row")
    return [_dequantise(*_quantise(v))[:, :v.shape[1]].to(dtype) for v in ways]


def _run_quantise_own(s):
    import fp8_block_scaled_dg_amd as dg
    x, way = s["x"], s["case"]["way"]
    if way == "both":
        q, sf, qt, sft = dg.to_mxfp4_both(x)
        return [dg.from_mxfp4(q, sf, x.shape[1], x.dtype), dg.from_mxfp4(qt, sft, x.shape[0], x.dtype)]
    q, sf = dg.to_mxfp4(x, transposed=way == "transposed")
    return [dg.from_mxfp4(q, sf, x.shape[way == "row"], x.dtype)]


def _product(a, sa, b, sb):
    return _dequantise(a, sa) @ _dequantise(b, sb).t()


def _run_linear(s):
    x, w, dy = s["x"], s["w"], s["dy"]
    y = _product(*_quantise(x), *_quantise(w))
    dx = _product(*_quantise(dy), *_quantise(w.t()))
    dw = _product(*_quantise(dy.t()), *_quantise(x.t()))
    return [v.to(torch.bfloat16) for v in (y, dx, dw)]


def _run_linear_own(s):
    import fp8_block_scaled_dg_amd as dg
    x, w, dy, ws = s["x"], s["w"], s["dy"], s["workspace"]
    qx, sx, qxt, sxt = dg.to_mxfp4_both(x)
    qw, sw, qwt, swt = dg.to_mxfp4_both(w)
    y = dg.mxfp4_gemm_nt(qx, qw, sx, sw, workspace=ws)
    qd, sd, qdt, sdt = dg.to_mxfp4_both(dy)
    return [y, dg.mxfp4_gemm_nt(qd, qwt, sd, swt, workspace=ws), dg.mxfp4_gemm_nt(qdt, qxt, sdt, sxt, workspace=ws)]


def _route(logits, k, scoring):
    v, ids = torch.sort(logits, dim=1, descending=True, stable=True)  # ties: lowest index first
    v, ids = v[:, :k], ids[:, :k]
    off = v == float("-inf")
    p = torch.softmax(logits, 1).gather(1, ids) if scoring == "softmax" else torch.sigmoid(v)
    p = torch.where(off, 0.0, p)
    p = p / p.sum(1, keepdim=True).clamp_min(1e-38)
    return torch.where(off, -1, ids).to(torch.int32), p


def _run_moe(s):
    case, x = s["case"], s["x"].float()
    T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
    values = _fp8_values if case["fmt"] == "fp8" else _dequantise
    ids, weights = _route(s["logits"], k, case["scoring"])
    share = torch.zeros(T, E + 1, device=x.device)  # the last column: slots that chose nothing
    share = share.scatter_add(1, torch.where(ids < 0, E, ids).long(), weights)[:, :E]
    gu = (x @ values(s["w13"], s["s13"]).reshape(E * 2 * I, H).t()).reshape(T, E, I, 2)
    gate, up = gu[..., 0], gu[..., 1]
    h = gate / (1.0 + torch.exp(-gate)) * up * share[..., None]
    y = h.reshape(T, E * I) @ values(s["w2"], s["s2"]).transpose(1, 2).reshape(E * I, H)
    return [y.to(torch.bfloat16), ids, weights]


def run(s):
    case = s["case"]
    kind = case["kind"]
    if kind == "quantise":
        return _run_quantise_own(s) if own else _run_quantise(s)
    if kind == "linear":
        return _run_linear_own(s) if own else _run_linear(s)
    if not own:
        if kind == "moe":
            return _run_moe(s)
        a = _dequantise(s["a"], s["sa"]) if kind == "product" else s["a"].float()
        return (a @ _dequantise(s["b"], s["sb"]).t()).to(torch.bfloat16)
    import fp8_block_scaled_dg_amd as dg
    if kind == "moe":
        dg.dg_moe_layer(s["y"], s["x"], s["w13"], s["w2"], s["s13"], s["s2"], s["ids"], s["weights"], logits=s["logits"], scoring=case["scoring"], workspace=s["workspace"])
        return [s["y"], s["ids"], s["weights"]]
    if kind == "a16":
        dg.dg_mxfp4_gemm_nt_bf16a(s["c"], s["a"], s["b"], s["sb"], workspace=s["workspace"])
    else:
        dg.dg_mxfp4_gemm_nt(s["c"], s["a"], s["b"], s["sa"], s["sb"], workspace=s["workspace"])
    return s["c"]


def work(case):
    """Inputs once, outputs once.  MXFP4 holds 32 values in 17 bytes."""
    kind, mx = case["kind"], 17 / 32
    if kind == "quantise":
        n, size, ways = case["rows"] * case["cols"], 2 if case["dtype"] == "bf16" else 4, 2 if case["way"] == "both" else 1
        # x read; per direction codes and scales written, read again, values written
        return {"bytes": n * (size + ways * (2 * mx + size)), "flops": 4 * n * ways}
    if kind in ("product", "a16"):
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * (mx if kind == "product" else 2) + N * K * mx + 2 * M * N, "flops": 2 * M * N * K}
    if kind == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        n = M * K + N * K + M * N
        # each operand read, both directions written and read, the three results written
        return {"bytes": n * (2 + 4 * mx + 2), "flops": 6 * M * N * K}
    T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
    touched = E * (1.0 - (1.0 - k / E) ** T)  # experts that T tokens reach, in the mean
    per = 1 + 4 / 128 ** 2 if case["fmt"] == "fp8" else mx
    return {"bytes": touched * 3 * H * I * per + 4 * T * H + 4 * T * E + 8 * T * k + 4 * T * k * I, "flops": 6 * T * k * H * I}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, apart from the above
# ---------------------------------------------------------------------------

def _round_mx64(x):
    """Every value of x [R][C] (float64) rounded to its block's MXFP4 grid."""
    R, C = x.shape
    full = -(-C // 32) * 32
    v = torch.zeros(R, full, dtype=torch.float64, device=x.device)
    v[:, :C] = x
    v = v.view(R, -1, 32)
    top = v.abs().max(-1, keepdim=True).values
    power = torch.frexp(top).exponent - 1  # floor(log2(top))
    power = torch.where(top > 0, power - 2, -127).clamp_min(-127).double()
    scale = torch.exp2(power)
    m = v.abs() / scale
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0)).double()
    m = (torch.round(m / step) * step).clamp_max(6.0)  # round: halves to even
    return (torch.copysign(m, v) * scale).view(R, full)[:, :C]


def _value64(q, sf):
    """MXFP4 codes [rows][bytes] and words -> float64, from the fields."""
    rows, n = q.shape
    nib = torch.stack((q & 15, q >> 4), -1).view(rows, 2 * n).long()
    ex, man = (nib >> 1) & 3, (nib & 1).double()
    mag = torch.where(ex == 0, man * 0.5, (1 + man * 0.5) * torch.exp2((ex - 1).double()))
    blk = torch.arange(2 * n, device=q.device) // 32
    word = sf.long()[blk // 4].t()  # [rows][K]
    byte = (word >> (8 * (blk % 4))) & 255
    v = torch.where(nib >= 8, -mag, mag) * torch.exp2(byte.double() - 127)
    return torch.where(byte == 255, float("nan"), v)


def _fp8_value64(codes, s):
    c = codes.long()
    ex, man = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(ex == 0, man / 8 * 2.0 ** -6, (1 + man / 8) * torch.exp2((ex - 7).double()))
    v = torch.where(c >= 128, -mag, mag)
    n, k = codes.shape
    sc = s.double()[torch.arange(k, device=s.device) // 128][:, torch.arange(n, device=s.device) // 128]
    return v * sc.t()


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "quantise":
        x = s["x"].double()
        ways = [x] * (case["way"] != "transposed") + [x.t()] * (case["way"] != "row")
        return [_round_mx64(v) for v in ways]
    if kind == "linear":
        x, w, dy = (s[n].double() for n in ("x", "w", "dy"))
        return [_round_mx64(x) @ _round_mx64(w).t(), _round_mx64(dy) @ _round_mx64(w.t().contiguous()).t(),
                _round_mx64(dy.t().contiguous()) @ _round_mx64(x.t().contiguous()).t()]
    if kind in ("product", "a16"):
        a = _value64(s["a"], s["sa"]) if kind == "product" else s["a"].double()
        return a @ _value64(s["b"], s["sb"]).t()
    T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
    value = _fp8_value64 if case["fmt"] == "fp8" else _value64
    l = s["logits"].double()
    score = torch.softmax(l, 1) if case["scoring"] == "softmax" else 1 / (1 + torch.exp(-l))
    order = torch.argsort(-l, dim=1, stable=True)[:, :k]
    w = score.gather(1, order)  # exactly 0 for an expert at -inf
    w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    x, y = s["x"].double(), torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = torch.nonzero((order == e) & (w > 0), as_tuple=True)
        if t.numel():
            gu = x[t] @ value(s["w13"][e], s["s13"][e]).t()
            h = gu[:, 0::2] * torch.sigmoid(gu[:, 0::2]) * gu[:, 1::2]
            y.index_add_(0, t, (h @ value(s["w2"][e], s["s2"][e]).t()) * w[t, j][:, None])
    return [y, None, w]
