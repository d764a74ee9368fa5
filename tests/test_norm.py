"""Residual addition with root-mean-square norm (moe_add_rmsnorm_fwd / _bwd), its
MXFP8 output and 8-bit checkpoint, and moe_mx_dequantize: refusals on the CPU, and
on the GPU the outputs against 64-bit formulas within derived bounds.

Bounds.  A sum of n fp32 terms of which no one passes through more than d additions
is off by at most d 2^-24 of the sum of magnitudes; the kernels' d is at most 32
(a thread's own values) + 6 (a wave) + 16 (waves) for a row.  rstd: half the
relative error of the mean, and three roundings more: 2^-18 covers it.  y and dx:
half a bf16 step, 2^-8 relative, and the fp32 terms before it."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import dispatch_grouped_gemm_moe_amd as moe
import oracle as O

FAKE = 1 << 20
EPS = 1e-5
ROW = 64 * 2.0 ** -24
HALF = 2.0 ** -8


# ------------------------------------------------------------------ refusals (no GPU)

def _fwd(rows=4, cols=64, eps=EPS, **over):
    a = dict(x=FAKE, res=None, w=FAKE, summed=None, y=2 * FAKE, rstd=None, yc=None, ys=None, cc=None, cs=None)
    a.update(over)
    return moe.lib().moe_add_rmsnorm_fwd(rows, cols, a["x"], a["res"], a["w"], eps, a["summed"], a["y"], a["rstd"],
                                         a["yc"], a["ys"], a["cc"], a["cs"], None)


@pytest.mark.parametrize("kw", [dict(rows=0), dict(rows=-1), dict(cols=0), dict(cols=48), dict(cols=-32),
                                dict(eps=-1.0), dict(eps=float("nan")), dict(x=None), dict(w=None), dict(y=None),
                                dict(x=FAKE + 8), dict(res=FAKE + 2), dict(w=FAKE + 4), dict(summed=FAKE + 8),
                                dict(y=FAKE + 8), dict(rstd=FAKE + 2), dict(yc=FAKE), dict(ys=FAKE), dict(cc=FAKE),
                                dict(cs=FAKE), dict(yc=FAKE + 8, ys=FAKE), dict(cc=FAKE, cs=FAKE + 1),
                                dict(summed=2 * FAKE)])
def test_norm_forward_refuses(kw):
    assert _fwd(**kw) == moe.MOE_E_INVALID


def test_norm_sizes_beyond_the_kernels():
    assert _fwd(cols=32800) == moe.MOE_E_UNSUPPORTED
    assert _fwd(rows=(1 << 21) + 1) == moe.MOE_E_UNSUPPORTED
    for rows, cols, want in ((0, 64, moe.MOE_E_INVALID), (4, 40, moe.MOE_E_INVALID), (4, 32800, moe.MOE_E_UNSUPPORTED)):
        with pytest.raises(moe.MoeError) as e:
            moe.moe_query_add_rmsnorm_bwd(rows, cols)
        assert e.value.status == want
    assert moe.lib().moe_query_add_rmsnorm_bwd(4, 64, None) == moe.MOE_E_INVALID


def _bwd(ws_bytes=1 << 30, rows=4, cols=64, **over):
    a = dict(dy=FAKE, dsum=None, s=FAKE, cc=None, cs=None, w=FAKE, rstd=FAKE, dx=FAKE, dw=FAKE, ws=FAKE)
    a.update(over)
    return moe.lib().moe_add_rmsnorm_bwd(rows, cols, a["dy"], a["dsum"], a["s"], a["cc"], a["cs"], a["w"], a["rstd"],
                                         a["dx"], a["dw"], a["ws"], ws_bytes, None)


@pytest.mark.parametrize("kw", [dict(dy=None), dict(w=None), dict(rstd=None), dict(dx=None), dict(dw=None),
                                dict(ws=None), dict(s=None), dict(cc=FAKE, cs=FAKE), dict(s=None, cc=FAKE),
                                dict(s=None, cs=FAKE), dict(dy=FAKE + 8), dict(dsum=FAKE + 8), dict(dx=FAKE + 2),
                                dict(dw=FAKE + 4), dict(ws=FAKE + 8), dict(rows=0), dict(cols=33)])
def test_norm_backward_refuses(kw):
    assert _bwd(**kw) == moe.MOE_E_INVALID


def test_norm_backward_refuses_a_small_workspace():
    assert _bwd(ws_bytes=moe.moe_query_add_rmsnorm_bwd(4, 64) - 1) == moe.MOE_E_WORKSPACE


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), moe.MOE_E_INVALID), (dict(cols=40), moe.MOE_E_INVALID), (dict(lay=2), moe.MOE_E_INVALID),
    (dict(c=None), moe.MOE_E_INVALID), (dict(s=None), moe.MOE_E_INVALID), (dict(d=None), moe.MOE_E_INVALID),
    (dict(c=FAKE + 8), moe.MOE_E_INVALID), (dict(d=FAKE + 8), moe.MOE_E_INVALID),
    (dict(rows=1 << 30, cols=32), moe.MOE_E_UNSUPPORTED)])
def test_dequantize_refuses(kw, want):
    a = dict(c=FAKE, s=FAKE, rows=4, cols=64, lay=0, d=FAKE)
    a.update(kw)
    assert moe.lib().moe_mx_dequantize(a["c"], a["s"], a["rows"], a["cols"], a["lay"], a["d"], None) == want


def test_norm_binding_refuses_tensors_the_kernels_cannot_read():
    b16 = torch.bfloat16
    x, w, y = torch.zeros(4, 64, dtype=b16), torch.zeros(64), torch.zeros(4, 64, dtype=b16)
    for kw in (dict(x=torch.zeros(64, 4, dtype=b16).t()), dict(x=torch.zeros(4, 64)), dict(weight=w.to(b16)),
               dict(y=y[:3]), dict(residual=torch.zeros(4, 128, dtype=b16)[:, ::2]), dict(rstd=torch.zeros(3)),
               dict(y_codes=torch.zeros(4, 64, dtype=torch.int8)), dict(y=y.to("meta"))):
        with pytest.raises(moe.MoeError) as e:
            moe.moe_add_rmsnorm_fwd(**{**dict(x=x, weight=w, y=y, stream=0), **kw})
        assert e.value.status == moe.MOE_E_INVALID


@pytest.mark.parametrize("rows,cols", [(4, (1 << 32) + 64), (4, 1 << 31), ((1 << 64) + 4, 64), (1 << 63, 64)])
def test_sizes_that_the_c_types_cannot_hold(rows, cols):
    with pytest.raises(moe.MoeError) as e:
        moe.moe_query_add_rmsnorm_bwd(rows, cols)
    assert e.value.status == moe.MOE_E_UNSUPPORTED


def test_tensors_of_more_columns_than_the_c_types_hold():
    # (meta tensors hold no memory; of any other size they are refused as not on a GPU)
    n = (1 << 32) + 64  # as an int32: 64
    big = lambda dtype: torch.empty(1, n, dtype=dtype, device="meta")
    b16, u8, gain = big(torch.bfloat16), big(torch.uint8), torch.empty(n, device="meta")
    one = torch.empty(1, device="meta")
    calls = [lambda: moe.moe_add_rmsnorm_fwd(b16, gain, b16, stream=0),
             lambda: moe.moe_add_rmsnorm_bwd(b16, gain, one, b16, gain, u8, summed=b16, stream=0),
             lambda: moe.moe_mx_dequantize(u8, u8, b16, stream=0),
             lambda: moe.moe_mx_quantize(b16, u8, u8, stream=0)]
    for call in calls:
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.status == moe.MOE_E_UNSUPPORTED


@pytest.mark.skipif(torch.cuda.is_available(), reason="the sizes that are not refused would be launched")
@pytest.mark.parametrize("cols", [32, 96, 7168, 32800])
def test_dequantize_refuses_2_to_the_35_codes_and_no_fewer(cols):
    most = ((1 << 35) - 1) // cols
    call = lambda rows: moe.lib().moe_mx_dequantize(FAKE, FAKE, rows, cols, 0, FAKE, None)
    assert call(most) == moe.MOE_E_HIP  # past every check; there is no GPU
    assert call(most + 1) == moe.MOE_E_UNSUPPORTED


# ------------------------------------------------------------------ GPU

COLS = [32, 64, 96, 128, 224, 512, 544, 1024, 1056, 2080, 4096, 4128, 7168, 8192, 8224, 16384, 32768]


def _rand(g, *shape, sigma=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g) * sigma).to(dtype).cuda()


def _norm_inputs(rows, cols, seed):
    g = torch.Generator().manual_seed(seed)
    x, r = _rand(g, rows, cols), _rand(g, rows, cols, sigma=4.0)
    w = 1 + _rand(g, cols, sigma=0.1, dtype=torch.float32)
    return g, x, r, w


def _forward(x, w, residual=None, codes=False, checkpoint=False, summed=None, y=None):
    """The forward with guard rows behind every output, as a dict of tensors."""
    rows, cols = x.shape

    def out(*shape, dtype):
        t = torch.full((shape[0] + 1, *shape[1:]), 77, dtype=dtype, device="cuda")
        guards.append(t)
        return t[:-1]

    guards = []
    o = {"y": out(rows, cols, dtype=torch.bfloat16) if y is None else y, "rstd": out(rows, dtype=torch.float32)}
    o["summed"] = out(rows, cols, dtype=torch.bfloat16) if summed is None else summed
    if codes:
        o["y_codes"] = out(rows, cols, dtype=torch.uint8)
        o["y_scales"] = out((cols + 127) // 128, rows, 4, dtype=torch.uint8)
    if checkpoint:
        o["ck_codes"] = out(rows, cols, dtype=torch.uint8)
        o["ck_scales"] = out(rows, cols // 32, dtype=torch.uint8)
    moe.moe_add_rmsnorm_fwd(x, w, eps=EPS, residual=residual, **o)
    torch.cuda.synchronize()
    assert all((t[-1] == 77).all() for t in guards), "written past the last row"
    return o


def _row_scales(y_scales, cols):
    """Operand layout [groups, rows, 4] -> [rows, cols / 32]; the spare bytes must be zero."""
    s = y_scales.cpu().numpy().transpose(1, 0, 2).reshape(y_scales.shape[1], -1)
    assert not s[:, cols // 32:].any()
    return s[:, :cols // 32]


@pytest.mark.gpu
@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("rows", [1, 3, 130])
def test_norm_forward(gpu_lib, rows, cols):
    if rows * cols > 1 << 21:
        rows = 5
    g, x, r, w = _norm_inputs(rows, cols, rows * 7 + cols)
    for residual in (None, r):
        o = _forward(x, w, residual, codes=True, checkpoint=True)
        want = x if residual is None else (x.float() + r.float()).bfloat16()
        assert torch.equal(o["summed"], want)
        s = want.double()
        rstd = (s.square().mean(1) + EPS).rsqrt()
        assert ((o["rstd"].double() / rstd - 1).abs() <= 2.0 ** -18).all()
        y = s * rstd[:, None] * w.double()
        assert ((o["y"].double() - y).abs() <= y.abs() * (HALF + 2.0 ** -16)).all()
        # the codes are those of the rounded outputs, bit for bit
        for codes, scales, of in ((o["y_codes"], _row_scales(o["y_scales"], cols), o["y"]),
                                  (o["ck_codes"], o["ck_scales"].cpu().numpy(), want)):
            c, sc = O.mx_quantize(of.cpu(), axis=1)
            np.testing.assert_array_equal(scales, sc)
            np.testing.assert_array_equal(codes.cpu().numpy(), c)


@pytest.mark.gpu
def test_norm_forward_optional_outputs_and_aliases(gpu_lib):
    rows, cols = 9, 4128
    _, x, r, w = _norm_inputs(rows, cols, 5)
    want = _forward(x, w, r, codes=True, checkpoint=True)
    y = torch.empty_like(x)
    moe.moe_add_rmsnorm_fwd(x, w, y, eps=EPS, residual=r)  # neither the sum nor 1/rms is wanted
    torch.cuda.synchronize()
    assert torch.equal(y, want["y"])
    for summed_in, y_in in ((0, None), (1, None), (0, 1), (1, 0)):
        bufs = [x.clone(), r.clone()]
        o = _forward(bufs[0], w, bufs[1], codes=True, summed=bufs[summed_in],
                     y=None if y_in is None else bufs[y_in])
        for n in ("summed", "y", "rstd", "y_codes", "y_scales"):
            assert torch.equal(o[n], want[n]), (summed_in, y_in, n)


@pytest.mark.gpu
def test_norm_forward_zero_huge_and_spoilt_rows(gpu_lib):
    rows, cols = 6, 1056
    _, x, r, w = _norm_inputs(rows, cols, 6)
    want = _forward(x, w, r, codes=True)
    x2, r2 = x.clone(), r.clone()
    x2[1], r2[1] = 0, 0
    x2[3, 5] = float("nan")
    x2[4] = 1e18  # the squares' sum is 1e39: infinite in fp32, so 1/rms is 0
    o = _forward(x2, w, r2, codes=True)
    assert not o["y"][1].any() and not o["y_codes"][1].any() and (o["y_scales"][:, 1][:8] == 127).all()
    assert abs(o["rstd"][1].item() * EPS ** 0.5 - 1) < 1e-6
    assert torch.isnan(o["y"][3]).all()
    for i in (0, 2, 5):
        assert torch.equal(o["y"][i], want["y"][i]) and torch.equal(o["y_codes"][i], want["y_codes"][i])


@pytest.mark.gpu
@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("rows", [1, 2, 5, 30, 700])
def test_norm_backward(gpu_lib, rows, cols):
    if rows * cols > 1 << 21:
        rows = 21
    g, x, r, w = _norm_inputs(rows, cols, rows * 11 + cols)
    o = _forward(x, w, r, checkpoint=True)
    dy, ds = _rand(g, rows, cols), _rand(g, rows, cols)
    rstd = o["rstd"].double()[:, None]
    held = O.mx_dequantize(o["ck_codes"].cpu().numpy(), o["ck_scales"].cpu().numpy(), axis=1)
    ws = torch.empty(moe.moe_query_add_rmsnorm_bwd(rows, cols), dtype=torch.uint8, device="cuda")
    for ck, with_ds in itertools.product((False, True), (False, True)):
        dx = torch.full((rows + 1, cols), 77, dtype=torch.bfloat16, device="cuda")
        dw = torch.full((cols + 4,), 77.0, device="cuda")
        src = dict(ck_codes=o["ck_codes"], ck_scales=o["ck_scales"]) if ck else dict(summed=o["summed"])
        runs = []
        for _ in range(2):
            ws.random_(0, 256)
            moe.moe_add_rmsnorm_bwd(dy, w, o["rstd"], dx, dw, ws, dsum=ds if with_ds else None, **src)
            torch.cuda.synchronize()
            runs.append((dx.clone(), dw.clone()))
        assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
        assert (dx[-1] == 77).all() and (dw[cols:] == 77).all()
        s = torch.from_numpy(held).cuda() if ck else o["summed"].double()
        xhat = s * rstd
        gy = dy.double() * w.double()
        c, cm = (gy * xhat).mean(1, keepdim=True), (gy * xhat).abs().mean(1, keepdim=True)
        d = ds.double() if with_ds else torch.zeros_like(gy)
        want = d + rstd * (gy - xhat * c)
        mag = d.abs() + rstd * (gy.abs() + xhat.abs() * (cm + c.abs()))
        assert ((dx[:-1].double() - want).abs() <= HALF * want.abs() + 1.01 * ROW * mag).all()
        depth = (rows + 511) // 512 + 16
        assert ((dw[:cols].double() - (dy.double() * xhat).sum(0)).abs()
                <= depth * 2.0 ** -24 * 1.01 * (dy.double() * xhat).abs().sum(0)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(20000, 64), (9001, 128), (9000, 224), (4001, 512), (2100, 992)])
def test_norm_backward_of_many_narrow_rows(gpu_lib, rows, cols):
    # a workgroup takes several rows at once, several times
    test_norm_backward(gpu_lib, rows, cols)


@pytest.mark.gpu
def test_norm_backward_against_differences(gpu_lib):
    """The kernel's gradients against central differences of the forward in 64 bits, along random
    directions.  The forward is smooth: with a step of 1e-5 the difference quotient is off by under
    1e-8 of the second-order scale; the kernel's dx is off by half a bf16 step in each element."""
    rows, cols = 4, 160
    g, x, _, w = _norm_inputs(rows, cols, 9)
    o = _forward(x, w)
    dy, ds = _rand(g, rows, cols), _rand(g, rows, cols)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty(moe.moe_query_add_rmsnorm_bwd(rows, cols), dtype=torch.uint8, device="cuda")
    moe.moe_add_rmsnorm_bwd(dy, w, o["rstd"], dx, dw, ws, summed=x, dsum=ds)
    torch.cuda.synchronize()

    def loss(s, w):
        y = s * (s.square().mean(1, keepdim=True) + EPS).rsqrt() * w
        return (y * dy.double()).sum() + (s * ds.double()).sum()

    s, wd, h = x.double(), w.double(), 1e-5
    for i in range(5):
        v = torch.randn(rows, cols, generator=g, dtype=torch.float64).cuda()
        vw = torch.randn(cols, generator=g, dtype=torch.float64).cuda()
        num = (loss(s + h * v, wd) - loss(s - h * v, wd)) / (2 * h)
        assert (num - (dx.double() * v).sum()).abs() <= ((HALF + 1e-4) * dx.double().abs() * v.abs()).sum()
        num = (loss(s, wd + h * vw) - loss(s, wd - h * vw)) / (2 * h)
        assert (num - (dw.double() * vw).sum()).abs() <= 1e-4 * (dw.double().abs() * vw.abs()).sum()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(33, 4128), (9000, 96), (2500, 800), (600, 16416)])
def test_norm_backward_in_place(gpu_lib, rows, cols):
    g, x, r, w = _norm_inputs(rows, cols, 8)
    o = _forward(x, w, r)
    dy, ds = _rand(g, rows, cols), _rand(g, rows, cols)
    ws = torch.empty(moe.moe_query_add_rmsnorm_bwd(rows, cols), dtype=torch.uint8, device="cuda")
    want, dw = torch.empty_like(x), torch.empty_like(w)
    moe.moe_add_rmsnorm_bwd(dy, w, o["rstd"], want, dw, ws, summed=o["summed"], dsum=ds)
    for which in (0, 1):
        b = [dy.clone(), ds.clone()]
        dw2 = torch.empty_like(w)
        moe.moe_add_rmsnorm_bwd(b[0], w, o["rstd"], b[which], dw2, ws, summed=o["summed"], dsum=b[1])
        torch.cuda.synchronize()
        assert torch.equal(b[which], want) and torch.equal(dw2, dw)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(1, 32), (7, 160), (300, 512), (5, 7168)])
def test_dequantize_gives_the_codes_values(gpu_lib, rows, cols):
    g = torch.Generator().manual_seed(rows + cols)
    codes = torch.randint(0, 256, (rows, cols), generator=g, dtype=torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x38  # no NaN code
    scales = torch.randint(0, 247, (rows, cols // 32), generator=g, dtype=torch.uint8)  # finite in bf16
    want = torch.from_numpy(O.mx_dequantize(codes.numpy(), scales.numpy(), axis=1)).float().bfloat16()
    groups = (cols + 127) // 128
    operand = torch.zeros(rows, groups * 4, dtype=torch.uint8)
    operand[:, :cols // 32] = scales
    operand = operand.view(rows, groups, 4).transpose(0, 1).contiguous()
    for sc, lay in ((scales, False), (operand, True)):
        dst = torch.full((rows + 1, cols), 77, dtype=torch.bfloat16, device="cuda")
        moe.moe_mx_dequantize(codes.cuda(), sc.cuda(), dst, operand_scales=lay)
        torch.cuda.synchronize()
        assert torch.equal(dst[:-1].cpu().view(torch.int16), want.view(torch.int16))
        assert (dst[-1] == 77).all()


@pytest.mark.gpu
def test_dequantize_nan_and_the_quantisers_own_codes(gpu_lib):
    codes = torch.full((2, 32), 0x38, dtype=torch.uint8)
    codes[0, 3], codes[0, 4] = 0x7F, 0xFF
    dst = torch.empty(2, 32, dtype=torch.bfloat16, device="cuda")
    moe.moe_mx_dequantize(codes.cuda(), torch.tensor([[127], [255]], dtype=torch.uint8).cuda(), dst)
    got = dst.cpu()
    assert torch.isnan(got[0, 3:5]).all() and (got[0, 5:] == 1).all() and torch.isnan(got[1]).all()
    src = (torch.randn(40, 256) * torch.logspace(-30, 30, 40)[:, None]).bfloat16()
    c, s = torch.empty(40, 256, dtype=torch.uint8, device="cuda"), torch.empty(40, 8, dtype=torch.uint8, device="cuda")
    back = torch.empty(40, 256, dtype=torch.bfloat16, device="cuda")
    moe.moe_mx_quantize(src.cuda(), c, s)
    moe.moe_mx_dequantize(c, s, back)
    assert torch.equal(back.cpu().double(), torch.from_numpy(O.mx_roundtrip(src, axis=1)))


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [1024, 1056, 20480])
def test_norm_offsets_past_32_bits(gpu_lib, cols):
    """Rows are independent, so the last rows of more than 2^32 bytes give what they give alone; only
    the very last row has a gradient, so dw has one term to add up."""
    rows, n = min(1 << 21, (1 << 31) // cols + 5), 3
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-n:] = torch.randn(n, cols, generator=g, device="cuda").bfloat16()
    w = torch.randn(cols, generator=g, device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    ck, cs = torch.empty(rows, cols, dtype=torch.uint8, device="cuda"), torch.empty(rows, cols // 32, dtype=torch.uint8,
                                                                                   device="cuda")
    yq, ys = torch.empty_like(ck), torch.empty((cols + 127) // 128, rows, 4, dtype=torch.uint8, device="cuda")
    moe.moe_add_rmsnorm_fwd(x, w, y, eps=EPS, rstd=rstd, y_codes=yq, y_scales=ys, ck_codes=ck, ck_scales=cs)
    small = _forward(x[-n:].contiguous(), w, codes=True, checkpoint=True)
    assert torch.equal(y[-n:], small["y"]) and torch.equal(rstd[-n:], small["rstd"])
    assert torch.equal(yq[-n:], small["y_codes"]) and torch.equal(ys[:, -n:], small["y_scales"])
    assert torch.equal(ck[-n:], small["ck_codes"]) and torch.equal(cs[-n:], small["ck_scales"])
    back = torch.empty(n, cols, dtype=torch.bfloat16, device="cuda")
    moe.moe_mx_dequantize(ck, cs, y)
    moe.moe_mx_dequantize(small["ck_codes"], small["ck_scales"], back)
    assert torch.equal(y[-n:], back)
    moe.moe_mx_dequantize(yq, ys, y, operand_scales=True)
    moe.moe_mx_dequantize(small["y_codes"], small["y_scales"], back, operand_scales=True)
    assert torch.equal(y[-n:], back)
    dy = torch.zeros_like(x)
    dy[-1] = torch.randn(cols, generator=g, device="cuda").bfloat16()
    ws = torch.empty(moe.moe_query_add_rmsnorm_bwd(rows, cols), dtype=torch.uint8, device="cuda")
    for src, part in ((dict(summed=x), dict(summed=x[-n:].contiguous())),
                      (dict(ck_codes=ck, ck_scales=cs), dict(ck_codes=small["ck_codes"], ck_scales=small["ck_scales"]))):
        dw, dw_part, dx_part = torch.empty_like(w), torch.empty_like(w), torch.empty_like(back)
        moe.moe_add_rmsnorm_bwd(dy, w, rstd, y, dw, ws, **src)
        moe.moe_add_rmsnorm_bwd(dy[-n:].contiguous(), w, small["rstd"], dx_part, dw_part, ws, **part)
        torch.cuda.synchronize()
        assert torch.equal(y[-n:], dx_part) and torch.equal(dw, dw_part)


@pytest.mark.gpu
def test_norm_captured_and_replayed(gpu_lib):
    rows, cols = 600, 2080
    g, x, r, w = _norm_inputs(rows, cols, 12)
    dy = _rand(g, rows, cols)
    ws = torch.empty(moe.moe_query_add_rmsnorm_bwd(rows, cols), dtype=torch.uint8, device="cuda")
    o = _forward(x, w, r, codes=True)
    dx, dw = torch.empty_like(x), torch.empty_like(w)

    def step():
        moe.moe_add_rmsnorm_fwd(x, w, eps=EPS, residual=r, **o)
        moe.moe_add_rmsnorm_bwd(dy, w, o["rstd"], dx, dw, ws, summed=o["summed"], dsum=dy)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x.add_(0.5)
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (*o.values(), dx, dw)]
        for t in (*o.values(), dx, dw):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*o.values(), dx, dw), want)), i


@pytest.mark.gpu
def test_block_of_norm_and_few_token_layer(gpu_lib):
    """The two as a decode step runs them: the norm's codes go into the layer."""
    from few_reference import few_layer
    from moe_inputs import Workload, make_inputs
    for prec, H in (("mxfp8", 448), ("bf16", 256)):
        wl = Workload("block_" + prec, T=6, H=H, I=128, E=8, k=2, prec=prec, shared_expert=True, stream=9900)
        inp = make_inputs(wl)
        mx = prec == "mxfp8"
        cfg = moe.make_cfg(6, H, 128, 8, 2, prec=int(mx), flags=moe.MOE_F_SHARED_EXPERT)
        packed = torch.empty(moe.moe_query_sizes(cfg).packed_weights, dtype=torch.uint8, device="cuda")
        moe.moe_prepare_weights(cfg, *(t.cuda() for t in (inp.Wg, inp.Wu, inp.Wd)), packed,
                                *(t.cuda() for t in (inp.Wsg, inp.Wsu, inp.Wsd)))
        few_ws = torch.zeros(moe.moe_query_few(cfg), dtype=torch.uint8, device="cuda")
        g, _, r, w = _norm_inputs(6, H, 3)
        stream, Wr = r.clone(), inp.Wr.cuda()
        x = inp.x.cuda()
        for _ in range(3):  # blocks in a row: each adds the last one's output
            o = _forward(x, w, stream, codes=mx, summed=stream)
            x = torch.empty_like(x)
            moe.moe_layer_fwd_few(cfg, Wr, None, packed, o["y"], x, few_ws, x_codes=o.get("y_codes"),
                                  x_scales=o.get("y_scales"))
            inp.x = o["y"].cpu()
            ref, bound = few_layer(inp, 6)
            assert (np.abs(x.double().cpu().numpy() - ref) <= bound).all()


# ------------------------------------------------------------------ NaN of any payload

NAN_BITS = (-1, 0x7FFFFFFF, 0x7FC00000, -0x400000, 0x7FFF8000, -0x8000)


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [64, 544, 4128, 16416])
def test_norm_keeps_a_nan_whatever_its_payload(gpu_lib, cols):
    rows = 3
    g, x, r, w = _norm_inputs(rows, cols, 31)
    dy = _rand(g, rows, cols)
    ws = torch.empty(moe.moe_query_add_rmsnorm_bwd(rows, cols), dtype=torch.uint8, device="cuda")

    def back(w, rstd):
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        moe.moe_add_rmsnorm_bwd(dy, w, rstd, dx, dw, ws, summed=want["summed"])
        torch.cuda.synchronize()
        return dx, dw

    want = _forward(x, w, r)
    dx, dw = back(w, want["rstd"])
    for i, b in enumerate(NAN_BITS):
        # a gain: its column of y, every row of dx (each row's mean has it), no part of dweight
        bad = w.clone()
        bad.view(torch.int32)[5 + i] = b
        o = _forward(x, bad, r)
        keep = torch.arange(cols, device="cuda") != 5 + i
        assert torch.isnan(o["y"][:, 5 + i]).all() and torch.equal(o["y"][:, keep], want["y"][:, keep]), hex(b)
        dx_bad, dw_bad = back(bad, want["rstd"])
        assert torch.isnan(dx_bad).all() and torch.equal(dw_bad, dw), hex(b)
        # 1/rms of a row: that row of dx, and all of dweight
        rstd = want["rstd"].clone()
        rstd.view(torch.int32)[1] = b
        dx_bad, dw_bad = back(w, rstd)
        assert torch.isnan(dx_bad[1]).all() and torch.isnan(dw_bad).all(), hex(b)
        assert torch.equal(dx_bad[0], dx[0]) and torch.equal(dx_bad[2], dx[2])
    # a sum: both signs of bf16's own NaN patterns pass through
    bad = x.clone()
    bad.view(torch.int16)[1, :4] = torch.tensor([0x7FFF, -1, 0x7F81, -0x7F], dtype=torch.int16, device="cuda")
    o = _forward(bad, w, r)
    assert torch.isnan(o["summed"][1, :4]).all() and torch.isnan(o["y"][1]).all()
    assert torch.equal(o["y"][0], want["y"][0])


@pytest.mark.gpu
def test_norm_backward_workspace_of_any_type(gpu_lib):
    x, w = torch.ones(40, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64, device="cuda")
    got = []
    for dtype in (torch.uint8, torch.float32):
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        ws = torch.empty(moe.moe_query_add_rmsnorm_bwd(40, 64), dtype=torch.uint8, device="cuda").view(dtype)
        moe.moe_add_rmsnorm_bwd(x, w, torch.ones(40, device="cuda"), dx, dw, ws, summed=x)
        torch.cuda.synchronize()
        got.append((dx, dw))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
