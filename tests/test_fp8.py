"""The norm with an 8-bit output, the plain quantisation and the block-scaled product against their
definitions in 64 bits, and their refusals.

Tolerances.  e4m3 rounds by at most half a step: 2^-4 of the value, or 2^-10 of the scale below the
smallest normal value 2^-6 (steps of 2^-9).  The float32 work before it (the residual's sum, a mean
of up to 2^14 terms in a tree of warps, a reciprocal root, three products) stays below 2^-19 of the
value.  A product's float32 sums of n terms are off by at most n 2^-23 of the sum of the absolute
terms (2^-23, not 2^-24: the tensor core may truncate), n = 128 within a block and one per block.
"""
import ctypes

import pytest
import torch

import linear_attention_layer_causal_b200 as gdn
import ops_ref as ref

F32 = 2.0 ** -19


def randn(seed, *shape, dev="cuda"):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dev)


def check_quant(q, scale, v, exact_scale):
    """q and scale against the float64 values v that they stand for."""
    assert torch.allclose(scale.double(), exact_scale, rtol=F32, atol=0)
    s = ref.widen(scale.double(), v.shape[1])
    err = (q.double() * s - v).abs()
    bound = 2.0 ** -4 * v.abs() + 2.0 ** -10 * s + F32 * v.abs()
    assert float((err - bound).max()) <= 0
    # saturation: the largest element of each block is held as 448 or its neighbour 416
    big = torch.stack([q[:, i:i + 128].double().abs().amax(1) for i in range(0, v.shape[1], 128)], 1)
    assert ((big == 448) | (exact_scale <= ref.TINY)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,dim,groups,dtype,residual,offset", [
    (1, 8, 1, torch.float32, False, 0.0),
    (3, 120, 1, torch.bfloat16, True, 1.0),
    (5, 128, 1, torch.float32, True, 0.0),
    (9, 136, 1, torch.bfloat16, False, 1.0),
    (7, 264, 1, torch.float32, True, 1.0),
    (33, 1024, 1, torch.bfloat16, True, 0.0),
    (2, 1032, 1, torch.bfloat16, True, 0.0),
    (3, 2048, 1, torch.float32, True, 1.0),
    (3, 2056, 1, torch.bfloat16, False, 0.0),
    (4, 4104, 1, torch.float32, True, 1.0),
    (257, 8192, 1, torch.bfloat16, True, 1.0),
    (2, 8200, 1, torch.bfloat16, True, 1.0),
    (2, 16384, 1, torch.float32, True, 0.0),
    (6, 1024, 8, torch.bfloat16, True, 1.0),
    (3, 8192, 4, torch.float32, False, 0.0),
    (2, 40960, 2, torch.bfloat16, True, 0.0),
    (2500, 2560, 1, torch.bfloat16, True, 1.0),   # a block takes several rows
    (1100, 1536, 3, torch.bfloat16, False, 0.0),  # and several groups' parts
    (8000, 136, 1, torch.float32, True, 1.0),
    (1000, 8192, 1, torch.float32, True, 0.0),
])
def test_norm(rows, dim, groups, dtype, residual, offset):
    x, w = (3 * randn(rows + dim, rows, dim)).to(dtype), 0.3 * randn(dim, dim)
    r = (5 * randn(dim + 1, rows, dim)).to(dtype) if residual else None
    out = gdn.rmsnorm_fp8(x, w, residual=r, groups=groups, eps=1e-5, weight_offset=offset, return_y=True)
    e = ref.norm(x, w, r, groups, 1e-5, offset)
    check_quant(out["q"], out["scale"], e["v"], e["scale"])
    step = torch.finfo(dtype).eps / 2
    assert float(((out["y"].double() - e["v"]).abs() - (step + F32) * e["v"].abs()).max()) <= 0
    if residual:
        assert torch.equal(out["residual"], (x.float() + r.float()).to(dtype))
    else:
        assert "residual" not in out


@pytest.mark.gpu
@pytest.mark.parametrize("rows,dim,dtype", [(1, 8, torch.bfloat16), (5, 200, torch.float32), (17, 2048, torch.bfloat16),
                                            (3, 12288, torch.bfloat16)])
def test_quantize(rows, dim, dtype):
    x = randn(dim, rows, dim).to(dtype)
    q, s = gdn.quantize_fp8(x)
    check_quant(q, s, x.double(), ref.block_scale(x.double()))


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [256, 2304, 16512])
def test_quantize_special_blocks(dim):
    """Blocks of zeros, of subnormal values, with an infinity, with a NaN; the others stay as they were."""
    x = randn(3, 4, dim)
    plain_q, plain_s = gdn.quantize_fp8(x)
    x[0, :128] = 0
    x[1, :128] = 1e-39
    x[2, 5] = float("inf")
    x[3, 130] = float("nan")
    q, s = gdn.quantize_fp8(x)
    assert s[0, 0] == ref.TINY and (q[0, :128].float() == 0).all()
    # 1e-39 is 0.085 of the smallest scale
    assert s[1, 0] == ref.TINY and ((q[1, :128].double() * ref.TINY / 1e-39 - 1).abs() <= 2.0 ** -4).all()
    assert s[2, 0] == float("inf") and q[2, 5].float().isnan() and (q[2, :5].float() == 0).all()
    assert s[3, 1].isnan() and q[3, 128:256].float().isnan().all()
    same = torch.ones(4, dim, dtype=torch.bool, device="cuda")
    same[0, :128] = same[1, :128] = same[2, :128] = False
    same[3, 128:256] = False
    assert torch.equal(q.float()[same], plain_q.float()[same])
    same_s = torch.ones_like(s, dtype=torch.bool)
    same_s[0, 0] = same_s[1, 0] = same_s[2, 0] = same_s[3, 1] = False
    assert torch.equal(s[same_s], plain_s[same_s])


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [512, 9000 // 8 * 8, 20480])
def test_norm_in_place_and_strided(dim):
    """The residual updated in place, x a slice of wider rows, outputs into given buffers."""
    wide = randn(1, 6, dim + 64).bfloat16()
    x, r, w = wide[:, 32:32 + dim], randn(2, 6, dim).bfloat16(), randn(3, dim)
    e = ref.norm(x, w, r)
    keep = (x.float() + r.float()).bfloat16()
    q, s = torch.empty(6, dim, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(6, -(-dim // 128), device="cuda")
    out = gdn.rmsnorm_fp8(x, w, residual=r, residual_out=r, q=q, scale=s)
    assert out["q"] is q and out["scale"] is s and out["residual"] is r
    check_quant(q, s, e["v"], e["scale"])
    assert torch.equal(r, keep)


@pytest.mark.gpu
def test_norm_of_zero_rows_and_zero_values():
    assert gdn.rmsnorm_fp8(torch.zeros(0, 64, device="cuda"), torch.ones(64, device="cuda"))["q"].shape == (0, 64)
    out = gdn.rmsnorm_fp8(torch.zeros(2, 64, device="cuda"), torch.ones(64, device="cuda"), eps=0.0)
    assert out["q"].float().isnan().all() and out["scale"].isnan().all()  # 0 / 0, as the formula has it
    out = gdn.rmsnorm_fp8(torch.zeros(2, 64, device="cuda"), torch.ones(64, device="cuda"))
    assert (out["q"].float() == 0).all() and (out["scale"] == ref.TINY).all()


def operands(M, N, K, seed):
    a, sa = ref.quant(randn(seed, M, K), 1)
    w, sw = ref.quant(randn(seed + 1, N, K), 128)
    return a, sa, w, sw


def check_product(out, a, sa, w, sw):
    e, mag = ref.product(a, sa, w, sw)
    kb = -(-a.shape[1] // 128)
    step = 2.0 ** -8 if out.dtype == torch.bfloat16 else 0.0
    over = (out.double() - e).abs() - ((128 + kb + 4) * 2.0 ** -23 * mag + step * e.abs())
    assert float(over.max()) <= 0, f"{float(over.max()):.2e} over the bound"
    # each element's rounding is at most `step` of it, so the 2-norm's is too: the elements next above a
    # power of two come close to it (2^-8 / sqrt(3) on average there, 2^-9 / sqrt(3) next below one)
    rel = float((out.double() - e).norm() / e.norm())
    assert rel <= step + 2.0 ** -17, f"{rel:.2e} in the 2-norm"


SHAPES = [(1, 1, 16), (1, 128, 128), (2, 129, 144), (3, 257, 112), (5, 7, 4112), (16, 384, 1024), (17, 130, 272),
          (33, 1000, 512), (64, 127, 640), (65, 256, 2048), (127, 12, 128), (128, 128, 256), (129, 255, 1040),
          (1537, 3331, 400), (31, 300, 2064), (50, 1030, 1552), (2100, 2400, 128), (200, 640, 768), (257, 513, 384), (300, 1032, 144), (1, 4096, 2048), (8, 520, 8192)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product(M, N, K, dtype):
    a, sa, w, sw = operands(M, N, K, M + N + K)
    out = gdn.matmul_fp8(a, sa, w, sw, out_dtype=dtype)
    assert out.dtype == dtype and out.shape == (M, N)
    check_product(out, a, sa, w, sw)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(4, 136, 256), (40, 200, 1024), (300, 264, 512)])
def test_product_into_wider_rows(M, N, K):
    """The columns around the output stay as they were, at row strides with and without alignment."""
    a, sa, w, sw = operands(M, N, K, 5)
    for width, first in ((N + 16, 8), (N + 5, 0)):
        for dtype in (torch.bfloat16, torch.float32):
            buf = torch.full((M, width), 9.0, dtype=dtype, device="cuda")
            gdn.matmul_fp8(a, sa, w, sw, out=buf[:, first:first + N])
            check_product(buf[:, first:first + N], a, sa, w, sw)
            assert (buf[:, :first] == 9).all() and (buf[:, first + N:] == 9).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [3, 150])
def test_product_scale_ranges_and_special_values(M):
    """Scales from 2^-100 to 2^60 in one row, a row that is NaN, zero operands."""
    N, K = 140, 512
    a, sa, w, sw = operands(M, N, K, 8)
    sa[0] = torch.tensor([2.0 ** -100, 1.0, 2.0 ** 60, 2.0 ** -30], device="cuda")
    a[1] = torch.zeros(K, device="cuda").to(a.dtype)
    sa[2, 1] = float("nan")
    out = gdn.matmul_fp8(a, sa, w, sw, out_dtype=torch.float32)
    assert out[2].isnan().all() and (out[1] == 0).all()
    keep = torch.tensor([i for i in range(M) if i not in (1, 2)], device="cuda")
    check_product(out[keep], a[keep], sa[keep], w, sw)
    for dtype in (torch.bfloat16, torch.float32):
        b = a.clone()
        b.view(torch.uint8)[0, 7] = 0x7f  # a NaN element
        out = gdn.matmul_fp8(b, sa, w, sw, out_dtype=dtype)
        assert out[0].isnan().all() and (out[1] == 0).all()


@pytest.mark.gpu
def test_product_repeats_bit_for_bit_and_in_a_graph():
    """The same call gives the same bits, eagerly, on another stream and replayed, two graphs in turn."""
    graphs = []
    for M, N, K in ((1, 520, 4096), (190, 300, 1024)):
        a, sa, w, sw = operands(M, N, K, 9)
        first = gdn.matmul_fp8(a, sa, w, sw, out_dtype=torch.float32)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        other = gdn.matmul_fp8(a, sa, w, sw, out_dtype=torch.float32, stream=s)
        s.synchronize()
        assert torch.equal(first, other)
        ws = torch.empty(gdn.matmul_fp8_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
        out = torch.zeros_like(first)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gdn.matmul_fp8(a, sa, w, sw, out=out, workspace=ws)
        graphs.append((g, out, first, (a, sa, w, sw, ws)))  # a graph's operands have to live as long as it
    for _ in range(3):
        for g, out, *_rest in graphs:
            out.zero_()
            g.replay()
        torch.cuda.synchronize()
        for g, out, first, _kept in graphs:
            assert torch.equal(out, first)


@pytest.mark.gpu
def test_product_of_nothing():
    a, sa, w, sw = operands(4, 8, 32, 1)
    assert gdn.matmul_fp8(a[:0], sa[:0], w, sw).shape == (0, 8)
    assert gdn.matmul_fp8(a, sa, w[:0], sw[:0]).shape == (4, 0)


# ---------------------------------------------------------------- refusals

def test_binding_refusals_on_the_cpu():
    x, w = torch.zeros(2, 64), torch.zeros(64)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.rmsnorm_fp8(x, w)
    with pytest.raises(ValueError, match="weight"):
        gdn.rmsnorm_fp8(x, None)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        gdn.quantize_fp8(x.double())
    a = torch.zeros(2, 64, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.matmul_fp8(a, torch.zeros(2, 1), a, torch.zeros(1, 1))
    with pytest.raises(ValueError, match="out_dtype"):
        gdn.matmul_fp8(a, torch.zeros(2, 1), a, torch.zeros(1, 1), out_dtype=torch.float16)


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="argument-error cases run only without a GPU")
P = 1 << 20
I, U, W = gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_WORKSPACE


@no_gpu
def test_norm_abi_refusals():
    ok = dict(x=P, xs=256, res=P, w=P, ro=P, y=P, q=P, scale=P)

    def call(rows=4, dim=256, groups=1, eps=1e-6, off=0.0, dt=gdn.GDN_BF16, **over):
        cfg = gdn._NormConfig(rows, dim, groups, eps, off, dt)
        return gdn.lib().gdn_rmsnorm_fp8(ctypes.byref(cfg), *{**ok, **over}.values(), None)
    for over in (dict(rows=-1), dict(dim=0), dict(dim=252), dict(groups=0), dict(groups=3), dict(eps=-1.0),
                 dict(eps=float("nan")), dict(off=float("inf")), dict(dt=5), dict(x=None), dict(q=None), dict(scale=None),
                 dict(q=None, scale=None, y=None, ro=None), dict(xs=255), dict(xs=260), dict(x=P + 8), dict(res=P + 2),
                 dict(w=P + 4), dict(ro=P + 8), dict(y=P + 8), dict(q=P + 8), dict(scale=P + 2), dict(ro=P, x=P, xs=264)):
        assert call(**over) == I, over
    assert call(groups=4) == U and call(rows=1 << 31) == U and call(dim=1 << 25, xs=1 << 25) == U
    assert call(rows=0) == gdn.GDN_OK
    assert gdn.lib().gdn_rmsnorm_fp8(None, *ok.values(), None) == I


@no_gpu
def test_product_abi_refusals():
    ok = dict(a=P, sa=P, w=P, sw=P, M=4, N=8, K=32, out=P, os=8, dt=0, ws=P, wsb=1 << 30)

    def call(**over):
        return gdn.lib().gdn_matmul_fp8(*{**ok, **over}.values(), None)
    for over in (dict(K=0), dict(K=24), dict(K=-16), dict(M=-1), dict(N=-1), dict(dt=7), dict(a=None), dict(sa=None),
                 dict(w=None), dict(sw=None), dict(out=None), dict(os=7), dict(os=1 << 40), dict(a=P + 8), dict(w=P + 1),
                 dict(out=P + 8), dict(sa=P + 2), dict(sw=P + 2)):
        assert call(**over) == I, over
    assert call(M=1 << 31) == U and call(N=1 << 31) == U and call(K=1 << 31) == U
    assert call(M=0) == gdn.GDN_OK and call(N=0) == gdn.GDN_OK
    n = ctypes.c_size_t(0)
    assert gdn.lib().gdn_matmul_fp8_workspace_size(4, 8, 24, ctypes.byref(n)) == I
    assert gdn.lib().gdn_matmul_fp8_workspace_size(4, 8, 32, None) == I
    need = gdn.matmul_fp8_workspace_size(1, 520, 8192)
    if need:
        big = dict(M=1, N=520, K=8192, os=520)
        assert call(**big, wsb=need - 1) == W and call(**big, ws=None) == W and call(**big, ws=P + 4) == W


@pytest.mark.gpu
def test_binding_refuses_wrong_shapes_types_and_strides():
    x, w = torch.zeros(2, 256, device="cuda"), torch.zeros(256, device="cuda")
    for kw in (dict(residual=x.bfloat16()), dict(residual=x[:, :128]), dict(q=torch.empty(2, 256, device="cuda")),
               dict(scale=torch.empty(2, 3, device="cuda")), dict(y=x.T)):
        with pytest.raises(ValueError):
            gdn.rmsnorm_fp8(x, w, **kw)
    with pytest.raises(ValueError):
        gdn.rmsnorm_fp8(x, w[:128])
    with pytest.raises(ValueError):
        gdn.rmsnorm_fp8(torch.zeros(256, 4, device="cuda").T, w)
    with pytest.raises(gdn.GdnError):
        gdn.rmsnorm_fp8(x, w, groups=4)
    a, sa, b, sb = operands(4, 8, 160, 1)
    for bad in ((a.float(), sa, b, sb), (a, sa[:, :1], b, sb), (a, sa, b[:, :144], sb), (a, sa, b, sb[:, :1]),
                (a, sa.cpu(), b, sb), (a, sa, b, sb.double()), (a[:, ::2], sa, b, sb)):
        with pytest.raises(ValueError):
            gdn.matmul_fp8(*bad)
    with pytest.raises(ValueError):
        gdn.matmul_fp8(a, sa, b, sb, out=torch.empty(4, 9, device="cuda"))


@pytest.mark.gpu
def test_past_32_bit_offsets():
    """Rows whose offsets pass 2^31 elements give what they give alone."""
    rows, dim = 300000, 8192
    assert rows * dim > 2 ** 31
    x = torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda")
    x[-3:] = randn(60, 3, dim).bfloat16()
    w = randn(61, dim)
    out, alone = gdn.rmsnorm_fp8(x, w), gdn.rmsnorm_fp8(x[-3:], w)
    assert torch.equal(out["q"][-3:].view(torch.uint8), alone["q"].view(torch.uint8))
    assert torch.equal(out["scale"][-3:], alone["scale"])
    del x
    a, sa, wq, sw = operands(300, 12352, 128, 62)
    M = 180000
    assert M * 12352 > 2 ** 31
    big = torch.zeros(M, 128, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.zeros(M, 1, device="cuda")
    big.view(torch.uint8)[-300:] = a.view(torch.uint8)
    scales[-300:] = sa
    assert torch.equal(gdn.matmul_fp8(big, scales, wq, sw)[-300:], gdn.matmul_fp8(a, sa, wq, sw))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 300])
def test_two_streams_and_status_words(M):
    """Products that overlap, with workspaces of their own; a given one comes back with clear status words."""
    a, sa, w, sw = operands(M, 1000, 2048, 63)
    want = gdn.matmul_fp8(a, sa, w, sw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [gdn.matmul_fp8(a, sa, w, sw, stream=s) for _ in range(6) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    ws = torch.full((gdn.matmul_fp8_workspace_size(M, 1000, 2048),), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(gdn.matmul_fp8(a, sa, w, sw, workspace=ws), want)
    assert (ws[:8] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 8192, 8192), (100, 4096, 4096), (3000, 4096, 4096)])
def test_a_wait_that_runs_out_is_reported(M, N, K):
    """With a bound of a few cycles on the waits between warps the call ends, says so, and the next one is whole."""
    a, sa, w, sw = operands(M, N, K, 64)
    ws = torch.empty(gdn.matmul_fp8_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    want = gdn.matmul_fp8(a, sa, w, sw, workspace=ws)
    assert gdn.prefill_status(ws) == (gdn.GDN_OK, 0)
    gdn.wait_limit_next_call(1)
    gdn.matmul_fp8(a, sa, w, sw, workspace=ws)
    assert gdn.prefill_status(ws)[0] == gdn.GDN_ERR_TIMEOUT
    assert torch.equal(gdn.matmul_fp8(a, sa, w, sw, workspace=ws), want)
    assert gdn.prefill_status(ws) == (gdn.GDN_OK, 0)
