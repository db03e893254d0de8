"""The MXFP4 and layer entry points of the binding refuse wrong arguments as the
older ones do: TypeError for a wrong type, ValueError for a wrong shape, layout
or device, DGError for what the library refuses.  Nothing is launched, so the
outputs stay as they were."""
import pytest
import torch

from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    need_gpu()
    import fp8_block_scaled_dg_amd as m
    return m


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8, device="cuda")


def i32(*s):
    return torch.zeros(s, dtype=torch.int32, device="cuda")


def bf(*s):
    return torch.full(s, 7.0, dtype=torch.bfloat16, device="cuda")


def refused(error, fn, *args, **kw):
    with pytest.raises(error):
        fn(*args, **kw)


def test_product(dg):
    c, a, b, sa, sb = bf(4, 6), u8(4, 64), u8(6, 64), i32(1, 4), i32(1, 6)
    f = dg.dg_mxfp4_gemm_nt
    for wrong in (None, 3, a.cpu().numpy()):
        refused(TypeError, f, c, wrong, b, sa, sb)
        refused(TypeError, f, c, a, wrong, sa, sb)
        refused(TypeError, f, c, a, b, wrong, sb)
        refused(TypeError, f, c, a, b, sa, wrong)
        refused(TypeError, f, wrong, a, b, sa, sb)
        refused(TypeError, dg.mxfp4_gemm_nt, wrong, b, sa, sb)
        refused(TypeError, dg.mxfp4_gemm_nt, a, wrong, sa, sb)
    refused(TypeError, f, c, a.float(), b, sa, sb)
    refused(TypeError, f, c.float(), a, b, sa, sb)
    refused(TypeError, f, c, a, b, sa.float(), sb)
    for bad in (a[0], a[None], a[:3], u8(4, 48), a.cpu(), u8(64, 4).t()):
        refused(ValueError, f, c, bad, b, sa, sb)
    for bad in (b[0], b[None], b[:5], u8(6, 48), b.cpu(), u8(64, 6).t()):
        refused(ValueError, f, c, a, bad, sa, sb)
    for bad in (sa[0], i32(2, 4), i32(1, 5), sa.cpu()):
        refused(ValueError, f, c, a, b, bad, sb)
    for bad in (c[0], c[:, :5], bf(6, 4), bf(6, 4).t(), c.cpu()):
        refused(ValueError, f, bad, a, b, sa, sb)
    refused(ValueError, f, c, a, b, sa, sb, workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    # K % 32, a short workspace
    refused((ValueError, dg.DGError), f, c, u8(4, 8), u8(6, 8), sa, sb)
    M, N, K = 16, 1024, 16384
    need = dg.dg_mxfp4_gemm_nt_workspace_bytes(M, N, K)
    refused(dg.DGError, f, bf(M, N), u8(M, K // 2), u8(N, K // 2), i32(K // 128, M), i32(K // 128, N),
            workspace=u8(need - 16))
    assert bool((c == 7).all())


def test_product_bf16a(dg):
    c, a, b, sb = bf(4, 6), bf(4, 128), u8(6, 64), i32(1, 6)
    f = dg.dg_mxfp4_gemm_nt_bf16a
    for wrong in (None, 3):
        refused(TypeError, f, c, wrong, b, sb)
        refused(TypeError, f, c, a, wrong, sb)
        refused(TypeError, f, c, a, b, wrong)
    for bad in (a[0], a[None], a[:3], bf(4, 96), bf(128, 4).t(), a.cpu()):
        refused(ValueError, f, c, bad, b, sb)
    for bad in (b[0], b[None], b[:5], u8(6, 48)):
        refused(ValueError, f, c, a, bad, sb)
    refused(dg.DGError, f, bf(65, 6), bf(65, 128), b, sb)
    assert bool((c == 7).all())


def test_quantiser(dg):
    x = bf(8, 64)
    for wrong in (None, 3, x.half(), x.int()):
        refused(TypeError, dg.to_mxfp4, wrong)
        refused(TypeError, dg.to_mxfp4_both, wrong)
    for bad in (x[0], x[None], x.t(), x[:1].expand(8, 64), x.cpu()):
        refused(ValueError, dg.to_mxfp4, bad)
    q, sf = dg.to_mxfp4(x)
    for wrong in (None, 3, q.float()):
        refused(TypeError, dg.from_mxfp4, wrong, sf, 64)
    refused(TypeError, dg.from_mxfp4, q, None, 64)
    for bad in (q[0], q[None], q[:7], q.cpu()):
        refused(ValueError, dg.from_mxfp4, bad, sf, 64)
    refused(ValueError, dg.from_mxfp4, q, sf, 65)
    refused(ValueError, dg.dg_quantize_mxfp4, x, q[:7], sf)
    refused(TypeError, dg.dg_quantize_mxfp4, x, q, None)
    refused(dg.DGError, dg.dg_quantize_mxfp4, x)


def test_layer(dg):
    T, E, k, H, I = 2, 3, 2, 64, 32
    good = dict(y=bf(T, H), x=bf(T, H), w13=u8(E, 2 * I, H // 2), w2=u8(E, H, I // 2), s13=i32(E, 1, 2 * I),
                s2=i32(E, 1, H), ids=i32(T, k), weights=torch.zeros(T, k, device="cuda"),
                workspace=dg.alloc_workspace(dg.dg_moe_layer_workspace_bytes(T, E, k, H, I)))

    def call(error, **kw):
        with pytest.raises(error):
            dg.dg_moe_layer(**dict(good, **kw))
    for name in ("y", "x", "w13", "w2", "s13", "s2", "ids", "weights"):
        t = good[name]
        for wrong in (None, 3, t.double()):
            call(TypeError, **{name: wrong})
        for bad in (t[0], t[None], t[:-1], t.cpu()):
            call(ValueError, **{name: bad})
        call(ValueError, **{name: torch.stack((t, t), -1)[..., 0]})
    call(ValueError, w13=u8(E))
    call(ValueError, ids=i32(T))
    call(ValueError, logits=torch.zeros(T, E + 1, device="cuda"))
    call(TypeError, logits=torch.zeros(T, E, device="cuda").double())
    call(dg.DGError, workspace=None)
    call(dg.DGError, workspace=good["workspace"][:-32].clone())
    assert bool((good["y"] == 7).all())
