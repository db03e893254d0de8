"""Routing, layout, dispatch, the grouped products, the 8-bit SwiGLU and combine
run together, forward and backward: every stage of the example against 64 bits
on what the stage read, the whole captured into graphs, and on other streams."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import moe_ref as ref
from gpu_util import assert_close, need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    need_gpu()
    import fp8_block_scaled_dg_amd as m
    return m


@pytest.fixture(scope="module")
def example(dg):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "moe_training_step.py")
    spec = importlib.util.spec_from_file_location("moe_training_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def f64(t):
    return t.double().cpu().numpy()


def fp8(q, s):
    return ref.values(q.cpu().numpy(), s.cpu().numpy())


def weights64(q, s):
    """codes [E, N, K] and 128 x 128 scales -> float64"""
    q, s = q.cpu().numpy(), f64(s)
    return np.stack([ref.e4m3(a) * np.repeat(np.repeat(b.T, 128, 0), 128, 1)[:a.shape[0]] for a, b in zip(q, s)])


def grouped64(a, w, mi):
    out = np.zeros((a.shape[0], w.shape[1]))
    for e in range(w.shape[0]):
        out[mi == e] = a[mi == e] @ w[e].T
    return out


@pytest.mark.parametrize("T,E,k", [(70, 5, 2), (1, 8, 3), (300, 2, 1)])
def test_every_stage_of_the_example(dg, example, T, E, k):
    args = ["--tokens", str(T), "--hidden", "384", "--inner", "256", "--experts", str(E), "--k", str(k)]
    layer, x, logits, bias, y, s, dy, g = example.main(args)
    p, l = s["plan"], f64(logits)
    kw = dict(scoring="sigmoid", scale=2.0)
    ids, w = ref.route(l, k, bias=f64(bias), **kw)
    assert np.array_equal(s["ids"].cpu().numpy(), ids)
    w = f64(s["weights"])
    for got, want in zip(p, ref.plan(ids, E, p.pairs.numel())):
        assert np.array_equal(got.cpu().numpy(), want)
    mi, rows = p.m_indices.cpu().numpy(), p.rows.cpu().numpy()
    real, used = mi >= 0, ref.blocks_used(mi)
    # forward
    a = fp8(s["a"], s["sa"])[real]
    pair = p.pairs.cpu().numpy()[real]
    ref.check_quantised(s["a"].cpu().numpy()[real], np.ascontiguousarray(s["sa"].cpu().numpy()[:, real]),
                        f64(x)[pair // k], np.zeros_like(a))
    w13, w2 = weights64(*layer.w13[:2]), weights64(*layer.w2[:2])
    kept = fp8(s["kept"], s["skept"])[real]
    gu = grouped64(a, w13, mi[real])
    # the checkpoint is of the BF16 gate/up rows: 2^-8 of them, and the product's FP32 sums
    err = 2.0 ** -7 * np.abs(gu) + 1e-3 * np.sqrt(np.mean(gu ** 2))
    ref.check_quantised(s["kept"].cpu().numpy()[real], np.ascontiguousarray(s["skept"].cpu().numpy()[:, real]), gu, err)
    c = grouped64(fp8(s["h"], s["sh"])[real], w2, mi[real])
    assert_close(f64(s["c"])[real], c)
    assert not s["c"][torch.from_numpy(~real).cuda()].any()
    t = f64(s["c"])[rows] * w[..., None]
    want, size = t.sum(1), np.abs(t).sum(1) * (k + 2) * ref.U
    assert np.all(np.abs(f64(y) - want) <= size + 2.0 ** -8 * (np.abs(want) + size))
    # backward
    d = f64(dy)
    full = np.zeros((len(mi), 384))
    full[real] = d[pair // k] * w.reshape(-1)[pair][:, None]
    ref.check_quantised(g["dc"].cpu().numpy()[real], np.ascontiguousarray(g["sdc"].cpu().numpy()[:, real]), full[real],
                        np.abs(full[real]) * 2 * ref.U)
    t = f64(s["c"])[rows] * d[:, None]
    assert np.all(np.abs(f64(g["dweights"]) - t.sum(-1)) <= np.abs(t).sum(-1) * 20 * ref.U)
    want, size = ref.route_gradient(l, ids, f64(g["dweights"]), scoring="sigmoid", scale=2.0)
    assert np.all(np.abs(f64(g["logits"]) - want) <= size * 400 * ref.U + 2.0 ** -126)
    dc = fp8(g["dc"], g["sdc"])[real]
    dh = f64(g["dh"])[real]
    assert_close(dh, grouped64(dc, w2.transpose(0, 2, 1), mi[real]))
    da, db, ea, eb = ref.swiglu_gradient(kept[:, 0::2], kept[:, 1::2], dh)
    ref.check_quantised(g["dgu"].cpu().numpy()[real], np.ascontiguousarray(g["sdgu"].cpu().numpy()[:, real]),
                        np.stack((da, db), -1).reshape(dh.shape[0], -1), np.stack((ea, eb), -1).reshape(dh.shape[0], -1))
    ref.check_quantised(g["h"].cpu().numpy()[real], np.ascontiguousarray(g["sh"].cpu().numpy()[:, real]),
                        *ref.swiglu(kept[:, 0::2], kept[:, 1::2]))
    dgu = fp8(g["dgu"], g["sdgu"])[real]
    assert_close(f64(g["rows"])[real], grouped64(dgu, w13.transpose(0, 2, 1), mi[real]))
    t = f64(g["rows"])[rows]
    want, size = t.sum(1), np.abs(t).sum(1) * (k + 2) * ref.U
    assert np.all(np.abs(f64(g["x"]) - want) <= size + 2.0 ** -8 * (np.abs(want) + size))
    # weight gradients: both operands are quantised anew along the rows, each value off by
    # 2^-4 of itself or 2^-10 of its block's scale, 2^-18.8 of the block's largest value
    h = fp8(g["h"], g["sh"])[real]
    for got, left, right in ((g["w2"], dc, h), (g["w13"], dgu, a)):
        for e in range(E):
            m = mi[real] == e
            L, R = left[m], right[m]
            eL, eR = ((2.0 ** -4 * np.abs(v) + 2.0 ** -18 * (np.abs(v).max() if v.size else 0.0)) for v in (L, R))
            want = L.T @ R
            bound = eL.T @ np.abs(R) + np.abs(L).T @ eR + eL.T @ eR
            sums = np.abs(L).T @ np.abs(R) * max(1, m.sum()) * 2 * ref.U
            assert np.all(np.abs(f64(got[e]) - want) <= bound + sums + 2.0 ** -8 * (np.abs(want) + bound))


def case(dg, T=70, E=6, k=2, H=256, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
    return x, torch.randn(T, E, device="cuda", generator=g), torch.randn(E, device="cuda", generator=g) * 0.1


def run_all(dg, x, logits, bias, ws):
    """Every entry point once, allocating nothing but outputs from torch."""
    T, H, k, E = x.shape[0], x.shape[1], 2, logits.shape[1]
    ids, w = dg.moe_route(logits, k, bias=bias, scoring="sigmoid", groups=2, top_groups=1, group_best=2)
    M = dg.dg_moe_plan_rows(T, E, k)
    i32 = dict(dtype=torch.int32, device="cuda")
    p = dg.MoePlan(torch.empty(T, k, **i32), torch.empty(M, **i32), torch.empty(M, **i32),
                   torch.empty(E + 1, dtype=torch.int64, device="cuda"), torch.empty(E, **i32))
    dg.dg_moe_plan(*p, ids, workspace=ws)
    zeros = lambda *s, **kw: torch.zeros(*s, device="cuda", **kw)
    a, sa = zeros(M, H, dtype=torch.uint8), zeros(H // 128, M)
    dg.dg_moe_dispatch_fp8(a, sa, x, p.rows, p.pairs)
    gu = zeros(M, H, dtype=torch.bfloat16)            # any rows will do: the tokens' own
    gu[p.rows.long().clamp_min(0).reshape(-1)] = x.repeat_interleave(k, 0)
    h, sh = zeros(M, H // 2, dtype=torch.uint8), zeros(H // 256, M)
    kept, skept = zeros(M, H, dtype=torch.uint8), zeros(H // 128, M)
    dg.dg_swiglu_fp8(h, sh, gu, kept, skept, m_indices=p.m_indices)
    y = dg.moe_combine(gu, p, w)
    dc, sdc, dw, dl = zeros(M, H, dtype=torch.uint8), zeros(H // 128, M), torch.empty_like(w), torch.empty_like(logits)
    dg.dg_moe_combine_backward(dc, sdc, dw, y, gu, p.rows, p.pairs, w)
    dg.dg_moe_route_backward(dl, dw, ids, logits, scoring="sigmoid")
    d, sd, dh = zeros(M, H, dtype=torch.uint8), zeros(H // 128, M), gu[:, :H // 2].contiguous()
    dg.dg_swiglu_fp8_backward(d, sd, dh, kept, skept, m_indices=p.m_indices)
    dt, sdt = zeros(H, M, dtype=torch.uint8), zeros(M // 128, H)
    dg.dg_transpose_fp8_blocks(dt, sdt, d, sd, block_rows=1, m_indices=p.m_indices)
    return [ids, w, *p, a, sa, h, sh, kept, skept, y, dc, sdc, dw, dl, d, sd, dt, sdt]


def same(got, want):
    for g, e in zip(got, want):
        assert torch.equal(g.view(torch.uint8), e.view(torch.uint8))


def test_graphs(dg):
    """Two graphs that share the plan's workspace, replayed in turn with new
    inputs and eager calls in between."""
    # 3000 pairs; the second graph's 9000 use the workspace
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    graphs = []
    for T in (1500, 4500):
        x, l, b = case(dg, T)
        run_all(dg, x, l, b, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = run_all(dg, x, l, b, ws)
        graphs.append((g, x, l, b, outs))
    for rep in range(3):
        for g, x, l, b, outs in graphs:
            nx, nl, nb = case(dg, x.shape[0], seed=10 + rep)
            x.copy_(nx), l.copy_(nl), b.copy_(nb)
            g.replay()
        torch.cuda.synchronize()
        for g, x, l, b, outs in graphs:
            same(outs, run_all(dg, x, l, b, ws))
        torch.cuda.synchronize()


def test_large_dispatch_in_a_graph(dg):
    """The workspace that a large call takes from torch, under capture."""
    T, E, k, H = 1030, 8, 8, 16384
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    ids = torch.randint(0, E, (T, k), device="cuda", dtype=torch.int32)
    p = dg.moe_plan(ids, E)
    assert dg.dg_moe_dispatch_fp8_workspace_bytes(T, k, H) > 0
    want = dg.moe_dispatch_fp8(x, p)
    used = p.m_indices.view(-1, 128)[:, 0].repeat_interleave(128) >= 0
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a, sa = dg.moe_dispatch_fp8(x, p)
    for _ in range(3):
        a.zero_(), sa.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a[used], want[0][used]) and torch.equal(sa[:, used], want[1][:, used])
        other = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")  # eager memory between replays
        del other


def test_two_streams_at_once(dg):
    """Calls with workspaces of their own on two streams give what each gives alone."""
    sets = [(case(dg, 4500, seed=s), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")) for s in (1, 2)]
    want = [run_all(dg, *c, ws) for c, ws in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run_all(dg, *sets[i][0], sets[i][1]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            same(g, want[i])


def test_explicit_stream(dg):
    x, l, b = case(dg)
    ids, w = dg.moe_route(l, 2)
    s = torch.cuda.Stream()
    i2, w2 = torch.empty_like(ids), torch.empty_like(w)
    s.wait_stream(torch.cuda.current_stream())
    dg.dg_moe_route(i2, w2, l, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(ids, i2) and torch.equal(w, w2)


def test_binding_refuses_on_the_device(dg):
    x, l, b = case(dg)
    ids, w = dg.moe_route(l, 2)
    p = dg.moe_plan(ids, 6)
    a, sa = dg.moe_dispatch_fp8(x, p)
    with pytest.raises(TypeError):
        dg.dg_moe_route(ids.long(), w, l)
    with pytest.raises(ValueError):
        dg.dg_moe_route(ids, w[:1], l)
    with pytest.raises(ValueError):
        dg.dg_moe_route(ids, w.t().contiguous().t(), l)
    with pytest.raises(ValueError):
        dg.dg_moe_route(ids, w, l, bias=b[:3])
    with pytest.raises(KeyError):
        dg.dg_moe_route(ids, w, l, scoring="tanh")
    with pytest.raises(ValueError):
        dg.dg_moe_route(ids, w, l.t())
    with pytest.raises(dg.DGError):
        dg.dg_moe_route(ids, w, l, groups=4)
    with pytest.raises(dg.DGError):
        dg.moe_route(l, 7)
    with pytest.raises(ValueError):
        dg.dg_moe_plan(p.rows, p.pairs, p.m_indices, p.offsets[:-1], p.counts, ids)
    with pytest.raises(dg.DGError):
        dg.dg_moe_plan(p.rows, p.pairs[:-128], p.m_indices[:-128], p.offsets, p.counts, ids)
    with pytest.raises(ValueError):
        dg.dg_moe_dispatch_fp8(a[:, :128], sa, x, p.rows, p.pairs)
    with pytest.raises(ValueError):
        dg.dg_moe_dispatch_fp8(a, sa.t(), x, p.rows, p.pairs)
    with pytest.raises(ValueError):
        dg.dg_moe_dispatch_fp8(a, sa.cpu(), x, p.rows, p.pairs)
    with pytest.raises(TypeError):
        dg.dg_moe_combine(x, x.float(), p.rows)
    with pytest.raises(ValueError):
        dg.dg_moe_combine(x, torch.zeros(256, 128, dtype=torch.bfloat16, device="cuda"), p.rows)
    with pytest.raises(ValueError):
        dg.dg_moe_combine_backward(a, sa, w, x, x, p.rows, p.pairs, w)
    with pytest.raises(TypeError):
        dg.dg_moe_combine_backward(a, None, None, x, None, p.rows, p.pairs, w)
    with pytest.raises(ValueError):
        dg.dg_swiglu_fp8(a, sa, x)
    with pytest.raises(dg.DGError):
        dg.swiglu_fp8(x[:, :128].contiguous())      # 64 hidden units
    with pytest.raises(ValueError):
        dg.dg_transpose_fp8_blocks(a, sa, a, sa)
    with pytest.raises(dg.DGError):
        dg.transpose_fp8_blocks(a[:100], sa[:, :100].contiguous())
