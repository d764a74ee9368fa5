"""8-bit floating point in blocks of 128 (moe_block_quantize, moe_block_quantize_weights,
moe_block_dequantize) and its products (moe_block_gemm, moe_block_gemm_swiglu): refusals on the CPU, and on
the GPU codes bit for bit and products against 64-bit sums.

Bounds of a product.  The matrix instruction cuts off what lies below 2^-13 of the largest of eight
neighbouring products: 8 * 2^-13 = 2^-10 of the sum of magnitudes at most.  The scaled additions in fp32 add
(blocks + 4) 2^-24 of it, and the output is rounded once (2^-8 of the value).  Codes that are whole numbers up
to 4 with scales that are powers of two leave nothing to cut off: their products are exact up to the last
rounding."""
import numpy as np
import pytest
import torch

import dispatch_grouped_gemm_moe_amd as moe

FAKE = 1 << 20
HALF = 2.0 ** -8
CUT = 2.0 ** -10


# ------------------------------------------------------------------ refusals (no GPU)

def _gemm(rows=4, n=64, k=64, groups=2, **over):
    a = dict(a=FAKE, sa=FAKE, off=FAKE, w=FAKE, sw=FAKE, out=FAKE)
    a.update(over)
    return moe.lib().moe_block_gemm(rows, n, k, groups, a["a"], a["sa"], a["off"], a["w"], a["sw"], a["out"], None)


def _swiglu(rows=4, n=64, k=64, groups=2, ws_bytes=1 << 30, **over):
    a = dict(a=FAKE, sa=FAKE, off=FAKE, wg=FAKE, sg=FAKE, wu=FAKE, su=FAKE, hq=FAKE, hs=FAKE, h=None, ws=FAKE)
    a.update(over)
    return moe.lib().moe_block_gemm_swiglu(rows, n, k, groups, a["a"], a["sa"], a["off"], a["wg"], a["sg"], a["wu"],
                                           a["su"], a["hq"], a["hs"], a["h"], a["ws"], ws_bytes, None)


SIZES = [dict(rows=0), dict(rows=-1), dict(n=0), dict(n=12), dict(k=0), dict(k=24), dict(k=-16), dict(groups=0),
         dict(off=None), dict(off=FAKE + 2), dict(a=None), dict(a=FAKE + 8), dict(sa=None), dict(sa=FAKE + 2)]
BIG = [dict(rows=(1 << 24) + 1), dict(groups=(1 << 16) + 1), dict(n=(1 << 20) + 16), dict(k=(1 << 20) + 16),
       dict(n=1 << 16, k=1 << 15)]


@pytest.mark.parametrize("kw", SIZES + [dict(w=None), dict(w=FAKE + 8), dict(sw=None), dict(sw=FAKE + 1),
                                        dict(out=None), dict(out=FAKE + 8)])
def test_product_refuses(kw):
    assert _gemm(**kw) == moe.MOE_E_INVALID


@pytest.mark.parametrize("kw", SIZES + [dict(n=72), dict(wg=None), dict(wu=None), dict(sg=None), dict(su=None),
                                        dict(wg=FAKE + 8), dict(wu=FAKE + 8), dict(sg=FAKE + 2), dict(su=FAKE + 2),
                                        dict(hq=None), dict(hs=None), dict(hq=FAKE + 8), dict(hs=FAKE + 2),
                                        dict(h=FAKE + 8), dict(ws=None), dict(ws=FAKE + 8)])
def test_swiglu_product_refuses(kw):
    assert _swiglu(**kw) == moe.MOE_E_INVALID


@pytest.mark.parametrize("kw", BIG)
def test_product_sizes_beyond_the_kernels(kw):
    assert _gemm(**kw) == moe.MOE_E_UNSUPPORTED
    assert _swiglu(**kw) == moe.MOE_E_UNSUPPORTED


def test_swiglu_workspace():
    need = moe.moe_query_block_swiglu(4, 64, 64, 2)
    assert _swiglu(ws_bytes=need - 1) == moe.MOE_E_WORKSPACE
    assert moe.lib().moe_query_block_swiglu(4, 64, 64, 2, None) == moe.MOE_E_INVALID
    for sizes, want in (((0, 64, 64, 2), moe.MOE_E_INVALID), ((4, 72, 64, 2), moe.MOE_E_INVALID),
                        ((4, 64, 64, 1 << 17), moe.MOE_E_UNSUPPORTED), ((4, 1 << 32, 64, 1), moe.MOE_E_UNSUPPORTED),
                        ((1 << 64, 64, 64, 1), moe.MOE_E_UNSUPPORTED)):
        with pytest.raises(moe.MoeError) as e:
            moe.moe_query_block_swiglu(*sizes)
        assert e.value.status == want


def test_swiglu_workspace_of_sizes_the_c_call_cannot_hold():
    """Their low bits alone would be sizes that it takes."""
    for sizes in ((4, 64 - (1 << 32), 64, 2), (4, 64, 64 - (1 << 32), 2), (4, 64, 64, 2 - (1 << 32)), (4 - (1 << 64), 64, 64, 2)):
        with pytest.raises(moe.MoeError) as e:
            moe.moe_query_block_swiglu(*sizes)
        assert e.value.status == moe.MOE_E_UNSUPPORTED


@pytest.mark.parametrize("n,k,groups", [(1024, 2048, 64), (2048, 7168, 32), (16, 13296, 26), (32, 3264, 1), (128, 128, 5),
                                        (144, 272, 256), (2048, 512, 600), (4096, 4096, 1), (528, 1040, 512)])
def test_a_swiglu_workspace_serves_fewer_rows(n, k, groups):
    """Sized once for the most rows of a batch: no smaller batch needs more."""
    most = 0
    for rows in sorted({int(1.05 ** i) for i in range(300)} | {4095, 4096, 4097, 24576, 131072, 1 << 24}):
        if rows > 1 << 24:
            break
        need = moe.moe_query_block_swiglu(rows, n, k, groups)
        assert need >= most, rows
        most = need


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), 1), (dict(cols=24), 1), (dict(cols=0), 1), (dict(src=None), 1), (dict(q=None), 1),
    (dict(s=None), 1), (dict(src=FAKE + 8), 1), (dict(q=FAKE + 8), 1), (dict(s=FAKE + 2), 1),
    (dict(rows=(1 << 30) + 1), 2), (dict(cols=(1 << 20) + 16), 2)])
def test_quantize_refuses(kw, want):
    a = dict(rows=4, cols=64, src=FAKE, q=FAKE, s=FAKE)
    a.update(kw)
    assert moe.lib().moe_block_quantize(a["rows"], a["cols"], a["src"], a["q"], a["s"], None) == want
    assert moe.lib().moe_block_dequantize(a["rows"], a["cols"], 0, a["src"], a["s"], a["q"], None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(g=0), 1), (dict(n=0), 1), (dict(n=12), 1), (dict(k=24), 1), (dict(t=2), 1), (dict(t=-1), 1),
    (dict(src=None), 1), (dict(q=None), 1), (dict(s=None), 1), (dict(src=FAKE + 8), 1), (dict(q=FAKE + 8), 1),
    (dict(s=FAKE + 2), 1), (dict(g=1 << 25), 2), (dict(n=1 << 20, k=1 << 11), 2), (dict(n=8, k=(1 << 20) + 16), 2)])
def test_quantize_weights_refuses(kw, want):
    a = dict(g=2, n=64, k=64, t=1, src=FAKE, q=FAKE, s=FAKE)
    a.update(kw)
    assert moe.lib().moe_block_quantize_weights(a["g"], a["n"], a["k"], a["src"], a["t"], a["q"], a["s"], None) == want


def test_dequantize_refuses_rows_that_are_no_whole_matrices():
    call = lambda rows, n: moe.lib().moe_block_dequantize(rows, 64, n, FAKE, FAKE, FAKE, None)
    assert call(10, 4) == call(10, -1) == moe.MOE_E_INVALID
    wide = moe.lib().moe_block_dequantize(8, (1 << 20) + 16, 8, FAKE, FAKE, FAKE, None)
    assert wide == moe.MOE_E_UNSUPPORTED  # more columns than the products and the kernel's grid take


def test_binding_refuses_tensors_the_kernels_cannot_read():
    u8, b16 = torch.uint8, torch.bfloat16
    a, sa = torch.zeros(4, 64, dtype=u8), torch.zeros(1, 4)
    w, sw = torch.zeros(2, 32, 64, dtype=u8), torch.zeros(2, 1, 1)
    off, out = torch.zeros(3, dtype=torch.int32), torch.zeros(4, 32, dtype=b16)
    good = dict(a=a, a_scales=sa, w=w, w_scales=sw, out=out, offsets=off, stream=0)
    bad = (dict(), dict(a=a.view(torch.int8)), dict(a_scales=sa[:, :3]), dict(a_scales=torch.zeros(1, 5)), dict(w=w[:, :, :32]), dict(w_scales=sw[:1]),
           dict(out=out[:3]), dict(out=out.float()), dict(offsets=off[:2]), dict(offsets=off.long()), dict(w=w.to("meta")))
    for kw in bad:
        with pytest.raises(moe.MoeError) as e:  # (the first: host tensors)
            moe.moe_block_gemm(**{**good, **kw})
        assert e.value.status == moe.MOE_E_INVALID
    good = dict(a=a, a_scales=sa, wg=w, wg_scales=sw, wu=w, wu_scales=sw, h_codes=torch.zeros(4, 32, dtype=u8),
                h_scales=torch.zeros(1, 4), ws=torch.zeros(4096, dtype=u8), offsets=off, stream=0)
    for kw in (dict(), dict(wu=w[:1]), dict(wu=w.reshape(2, 64, 32)), dict(wu_scales=sw[:1]), dict(a_scales=torch.zeros(1, 5)), dict(h=out[:3]), dict(h_scales=torch.zeros(1, 3)),
               dict(h_codes=torch.zeros(3, 32, dtype=u8))):
        with pytest.raises(moe.MoeError) as e:
            moe.moe_block_gemm_swiglu(**{**good, **kw})
        assert e.value.status == moe.MOE_E_INVALID


# ------------------------------------------------------------------ the quantisers (GPU)

def _exp(amax):
    """numpy: exponent of the scale of blocks with these largest magnitudes."""
    m, p = np.frexp(np.where(np.isfinite(amax), amax, 1.0).astype(np.float64))
    return np.where(amax > 0, np.maximum(p - 9 + (m > 0.875), -126), 0)


GRID = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()


def _code(v):
    """numpy: the E4M3 code nearest to v (|v| <= 448), a tie to the even code, by search."""
    a = np.abs(v)
    hi = np.searchsorted(GRID, a, side="left").clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = GRID[hi] - a, a - GRID[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(GRID[hi] == a, hi, code)
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def _row_codes(v):
    """numpy: codes and scales [blocks, rows] of v (float64 [rows, cols])."""
    rows, cols = v.shape
    codes, scales = np.empty((rows, cols), np.uint8), np.empty(((cols + 127) // 128, rows), np.float32)
    for b in range(scales.shape[0]):
        blk = v[:, 128 * b:128 * b + 128]
        e = _exp(np.abs(blk).max(1))
        codes[:, 128 * b:128 * b + 128] = _code(blk * 2.0 ** -e[:, None])
        scales[b] = 2.0 ** e
    return codes, scales


def _awkward(g, *shape):
    """bf16 values with borders of codes, blocks of zeros, one large value, the smallest and the largest."""
    v = torch.randn(*shape, generator=g) * torch.exp2(torch.randint(-20, 20, (shape[0], 1), generator=g).float())
    v = v.bfloat16()
    for i, x in ((1, 0.0), (2, 2.0 ** -133), (3, 3.3e38), (4, 448.0), (5, 1.0)):
        if i < shape[0]:
            v[i] = x
    if shape[0] > 6:
        v[6, ::2] = -(2.0 ** -130)
        v[6, 1] = 1.75
    return v


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 128), (7, 144), (9, 7168), (130, 512), (300, 48), (8, 2064),
                                       (5, 4112)])
def test_quantize_bit_for_bit(gpu_lib, rows, cols):
    v = _awkward(torch.Generator().manual_seed(rows + cols), rows, cols)
    nb = (cols + 127) // 128
    q = torch.full((rows + 1, cols), 77, dtype=torch.uint8, device="cuda")
    s = torch.full((nb * rows + 1,), 77.0, device="cuda")
    moe.moe_block_quantize(v.cuda(), q[:-1], s[:-1].view(nb, rows))
    codes, scales = _row_codes(v.double().numpy())
    np.testing.assert_array_equal(s[:-1].view(nb, rows).cpu().numpy(), scales)
    np.testing.assert_array_equal(q[:-1].cpu().numpy(), codes)
    assert (q[-1] == 77).all() and s[-1] == 77
    back = torch.full((rows + 1, cols), 77, dtype=torch.bfloat16, device="cuda")
    moe.moe_block_dequantize(q[:-1], s[:-1].view(nb, rows), back[:-1])
    want = q[:-1].cpu().view(torch.float8_e4m3fn).double() * torch.from_numpy(scales).double().t().repeat_interleave(128, 1)[:, :cols]
    assert torch.equal(back[:-1].cpu(), want.float().bfloat16()) and (back[-1] == 77).all()


@pytest.mark.gpu
@pytest.mark.parametrize("groups,n,k", [(1, 8, 16), (1, 128, 128), (3, 136, 144), (2, 264, 1040), (5, 64, 48), (1, 1000, 272)])
def test_quantize_weights_bit_for_bit(gpu_lib, groups, n, k):
    g = torch.Generator().manual_seed(groups * n + k)
    w = torch.stack([_awkward(g, n, k) for _ in range(groups)])
    if groups > 1:
        w[1] = 0
    nb, kb = (n + 127) // 128, (k + 127) // 128
    want_q, want_s = np.empty((groups, n, k), np.uint8), np.empty((groups, nb, kb), np.float32)
    v = w.double().numpy()
    for x in range(groups):
        for i in range(nb):
            for j in range(kb):
                blk = v[x, 128 * i:128 * i + 128, 128 * j:128 * j + 128]
                e = _exp(np.abs(blk).max())
                want_s[x, i, j] = 2.0 ** e
                want_q[x, 128 * i:128 * i + 128, 128 * j:128 * j + 128] = _code(blk * 2.0 ** -float(e))
    for transposed in (False, True):
        src = w.transpose(1, 2).contiguous() if transposed else w
        q = torch.full((groups * n * k + 16,), 77, dtype=torch.uint8, device="cuda")
        s = torch.full((groups * nb * kb + 1,), 77.0, device="cuda")
        qv, sv = q[:-16].view(groups, n, k), s[:-1].view(groups, nb, kb)
        moe.moe_block_quantize_weights(src.cuda(), qv, sv, transposed=transposed)
        np.testing.assert_array_equal(sv.cpu().numpy(), want_s)
        np.testing.assert_array_equal(qv.cpu().numpy(), want_q)
        assert (q[-16:] == 77).all() and s[-1] == 77
    back = torch.empty(groups, n, k, dtype=torch.bfloat16, device="cuda")
    moe.moe_block_dequantize(qv, sv, back, weights=True)
    sc = torch.from_numpy(want_s).double().repeat_interleave(128, 1)[:, :n].repeat_interleave(128, 2)[:, :, :k]
    want = torch.from_numpy(want_q).view(torch.float8_e4m3fn).double() * sc
    assert torch.equal(back.cpu(), want.float().bfloat16())


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(530001, 512), (1050003, 272), (2100001, 128)])
def test_quantize_many_rows(gpu_lib, rows, cols):
    """More rows than the grid has, past the last cache: as in pieces."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    v = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.bfloat16)
    nb, step = (cols + 127) // 128, 1 << 16
    q, s = torch.empty(rows, cols, dtype=torch.uint8, device="cuda"), torch.empty(nb, rows, device="cuda")
    moe.moe_block_quantize(v, q, s)
    for lo in range(0, rows, step):
        part = v[lo:lo + step]
        pq, ps = torch.empty_like(part, dtype=torch.uint8), torch.empty(nb, len(part), device="cuda")
        moe.moe_block_quantize(part, pq, ps)
        assert torch.equal(pq, q[lo:lo + step]) and torch.equal(ps, s[:, lo:lo + step])


@pytest.mark.gpu
def test_dequantize_past_32_bits(gpu_lib):
    """Values past 2^32 bytes, as rows and as matrices (one scale each for all blocks but the last row's)."""
    cols, n = 4112, 1024
    R = n * 511
    codes = (torch.arange(R * cols, dtype=torch.int64, device="cuda") % 126).to(torch.uint8).view(R, cols)
    codes[-1] += 128  # negative ones
    back = torch.empty(R, cols, dtype=torch.bfloat16, device="cuda")
    assert 2 * back.numel() > 1 << 32
    scales = torch.full((33, R), 2.0, device="cuda")
    scales[:, -1] = 0.5
    moe.moe_block_dequantize(codes, scales, back)
    table = torch.arange(256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).bfloat16()
    for lo in range(0, R, 1 << 16):
        part = codes[lo:lo + (1 << 16)]
        assert torch.equal(back[lo:lo + (1 << 16)], table[part.int()] * scales[0, lo:lo + (1 << 16), None].bfloat16())
    w = torch.full((511, n // 128, 33), 4.0, device="cuda")
    w[-1, -1] = 0.25
    moe.moe_block_dequantize(codes.view(511, n, cols), w, back.view(511, n, cols), weights=True)
    for lo in range(0, R, 1 << 16):
        part = codes[lo:lo + (1 << 16)]
        s = w[:, :, 0].reshape(-1).repeat_interleave(128)[lo:lo + (1 << 16), None]
        assert torch.equal(back[lo:lo + (1 << 16)], table[part.int()] * s.bfloat16())


@pytest.mark.gpu
def test_quantize_nan_and_infinity(gpu_lib):
    v = torch.ones(4, 256, dtype=torch.bfloat16)
    v[0, 3], v[1, 130], v[2, 7] = float("nan"), float("inf"), -float("inf")
    v.view(torch.int16)[3, 9] = 0x7fff
    q, s = torch.empty(4, 256, dtype=torch.uint8, device="cuda"), torch.empty(2, 4, device="cuda")
    moe.moe_block_quantize(v.cuda(), q, s)
    f = q.cpu().view(torch.float8_e4m3fn).float()
    for r, c in ((0, 3), (1, 130), (2, 7), (3, 9)):
        assert torch.isnan(f[r, c])
    assert (f[0, :3] * s[0, 0].item() == 1).all() and (f[1, :128] * s[0, 1].item() == 1).all()
    assert torch.isnan(f).sum() == 4


# ------------------------------------------------------------------ the products (GPU)

def _offsets(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)


def _operands(g, rows, k, groups, n, whole=False):
    """Codes and scales of both operands; whole: numbers whose sums are exact."""
    if whole:
        a = torch.randint(-4, 5, (rows, k), generator=g).to(torch.float8_e4m3fn)
        w = torch.randint(-2, 3, (groups, n, k), generator=g).to(torch.float8_e4m3fn)
    else:
        a = (torch.randn(rows, k, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
        w = (torch.randn(groups, n, k, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    sa = torch.exp2(torch.randint(-3, 4, ((k + 127) // 128, rows), generator=g).float())
    sw = torch.exp2(torch.randint(-3, 4, (groups, (n + 127) // 128, (k + 127) // 128), generator=g).float())
    if not whole:
        sa, sw = sa * (1 + torch.rand(sa.shape, generator=g)), sw * (1 + torch.rand(sw.shape, generator=g))
    return a, sa, w, sw


def _values(a, sa, w, sw):
    k, n = a.shape[1], w.shape[1]
    av = a.double() * sa.double().t().repeat_interleave(128, 1)[:, :k]
    wv = w.double() * sw.double().repeat_interleave(128, 1)[:, :n].repeat_interleave(128, 2)[:, :, :k]
    return av, wv


def _product(av, wv, offsets):
    """In 64 bits: the product by group, and the sum of its terms' magnitudes; NaN where there is no group."""
    out = torch.full((av.shape[0], wv.shape[1]), float("nan"), dtype=torch.float64, device=av.device)
    size = torch.zeros_like(out)
    for e in range(wv.shape[0]):
        lo, hi = offsets[e].item(), offsets[e + 1].item()
        out[lo:hi], size[lo:hi] = av[lo:hi] @ wv[e].t(), av[lo:hi].abs() @ wv[e].abs().t()
    return out, size


u8 = lambda t: t.view(torch.uint8).cuda()

# rows of each group, n, k
PRODUCTS = [([1], 8, 16), ([1], 64, 128), ([3], 264, 144), ([1, 0, 2], 136, 272), ([16], 128, 512), ([17], 128, 1040),
            ([0, 65, 0, 1, 130, 0], 256, 384), ([64, 64], 72, 256), ([300], 520, 400), ([257, 0, 255, 256, 1], 384, 656),
            ([5] * 70, 40, 144), ([0, 0, 0], 64, 64), ([700, 90], 1000, 1104), ([2, 1] * 40, 512, 2064), ([128], 248, 896),
            ([1024], 512, 128), ([40, 600], 776, 2576)]


def _uneven(rows, groups):
    """Counts that differ from group to group, some zero, some of whole tiles."""
    if groups == 1:
        return [rows]
    part = [(7 * i + 3) % 11 if i % 5 else 0 for i in range(groups)]
    counts = [rows * x // max(1, sum(part)) for x in part]
    counts[1 % groups] += -counts[1 % groups] % 256 if rows > 2000 else 0
    return counts


# rows, groups, n, k that fall to each of the forms in which the products are computed: tiles of 256 x 256,
# 128 x 256, 128 x 128, 64 x 256 and the few-row form, the first row past the tables of the tiles' groups
TILED = [(4100, 40, 1032, 144), (4100, 40, 1032, 400), (4100, 40, 1032, 656), (6100, 3, 2056, 272), (4129, 1, 4104, 272),
         (1500, 40, 1032, 144), (7000, 40, 264, 272), (2300, 40, 1032, 656), (2049, 1, 2056, 528), (100, 3, 6152, 400),
         (2300, 40, 264, 656), (1024, 1, 1032, 1040), (100, 40, 1032, 1040), (100, 40, 4104, 272), (300, 40, 1032, 400),
         (9000, 3, 2056, 144), (12000, 3, 4104, 272), (16400, 40, 2056, 144), (30000, 40, 1032, 656),
         (1300, 600, 136, 272), (12000, 600, 136, 272), (5000, 520, 40, 272)]
TILED_GLU = [(4100, 40, 528, 144), (4100, 40, 528, 400), (4100, 40, 528, 656), (4129, 1, 2064, 272), (1500, 40, 528, 144),
             (7000, 40, 144, 272), (7000, 40, 144, 656), (100, 40, 1552, 272), (100, 40, 528, 528), (700, 3, 1040, 656),
             (12000, 3, 2064, 272), (16400, 40, 1040, 144), (30000, 40, 528, 656), (1300, 600, 144, 272),
             (12000, 600, 144, 272)]
SHAPES = PRODUCTS + [(_uneven(r, e), n, k) for r, e, n, k in TILED]
SHAPES_GLU = [(c, (n + 15) // 16 * 16, k) for c, n, k in PRODUCTS] + [(_uneven(r, e), n, k) for r, e, n, k in TILED_GLU]
_name = lambda v: "x".join(map(str, [len(v), sum(v)])) if isinstance(v, list) else str(v)


@pytest.mark.gpu
@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("counts,n,k", SHAPES, ids=_name)
def test_product(gpu_lib, counts, n, k, whole):
    g = torch.Generator().manual_seed(sum(counts) + n + k)
    spare = 3  # rows of no group, left as they were
    rows, groups = sum(counts) + spare, len(counts)
    a, sa, w, sw = _operands(g, rows, k, groups, n, whole)
    off = _offsets(counts)
    want, size = (t.cpu() for t in _product(*_values(a.cuda(), sa.cuda(), w.cuda(), sw.cuda()), off))
    outs = []
    for _ in range(2):
        out = torch.full((rows + 1, n), 77, dtype=torch.bfloat16, device="cuda")
        moe.moe_block_gemm(u8(a), sa.cuda(), u8(w), sw.cuda(), out[:-1], offsets=off.cuda())
        torch.cuda.synchronize()
        outs.append(out.cpu())
    assert torch.equal(*outs)
    out, m = outs[0], sum(counts)
    assert (out[m:] == 77).all()
    if whole:
        assert torch.equal(out[:m], want[:m].float().bfloat16())
    else:
        assert ((out[:m].double() - want[:m]).abs() <= want[:m].abs() * HALF + size[:m] * CUT * 1.01).all()
        # As a whole far closer.  The roundings come to at most HALF of the norm.  What is cut off has either sign
        # alike: k terms of at most 2^-13 of a largest product (rms below 3 of the products' rms, of eight) come
        # to 3 * 2^-13 sqrt(k) of it, against a sum of sqrt(k): below 2^-11 = HALF / 8.
        assert (out[:m].double() - want[:m]).norm() <= want[:m].norm() * HALF * 1.125


@pytest.mark.gpu
@pytest.mark.parametrize("n,k", [(2112, 272), (2048, 640), (2056, 256)])
def test_output_past_the_last_cache(gpu_lib, n, k):
    """More than 2^28 bytes of output, of whole lines and not, by tiles of which most are whole: exact sums."""
    g = torch.Generator().manual_seed(n)
    counts = _uneven(70000, 3)
    rows = sum(counts) + 3
    a, sa, w, sw = _operands(g, rows, k, 3, n, True)
    off = _offsets(counts)
    a, sa, w, sw = a.cuda(), sa.cuda(), w.cuda(), sw.cuda()
    av, wv = _values(a, sa, w, sw)
    out = torch.full((rows, n), 77, dtype=torch.bfloat16, device="cuda")
    moe.moe_block_gemm(a.view(torch.uint8), sa, w.view(torch.uint8), sw, out, offsets=off.cuda())
    for e in range(3):
        lo, hi = off[e].item(), off[e + 1].item()
        assert torch.equal(out[lo:hi], (av[lo:hi] @ wv[e].t()).float().bfloat16())
    assert (out[sum(counts):] == 77).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,n,k", [(1, 64, 128), (37, 200, 336), (300, 264, 512)])
def test_product_of_one_group_needs_no_offsets(gpu_lib, rows, n, k):
    g = torch.Generator().manual_seed(rows)
    a, sa, w, sw = _operands(g, rows, k, 1, n)
    outs = []
    for off in (None, _offsets([rows]).cuda()):
        outs.append(torch.empty(rows, n, dtype=torch.bfloat16, device="cuda"))
        moe.moe_block_gemm(u8(a), sa.cuda(), u8(w), sw.cuda(), outs[-1], offsets=off)
    assert torch.equal(*outs)


@pytest.mark.gpu
@pytest.mark.parametrize("counts,n,k", SHAPES_GLU, ids=_name)
def test_swiglu_product(gpu_lib, counts, n, k):
    g = torch.Generator().manual_seed(sum(counts) + n + k + 1)
    spare = 2
    rows, groups, m = sum(counts) + spare, len(counts), sum(counts)
    a, sa, wg, sg = _operands(g, rows, k, groups, n)
    _, _, wu, su = _operands(g, 1, k, groups, n)
    # gate products of a size that silu bends
    sg, su = sg / (1e4 * k ** 0.5), su / (1e4 * k ** 0.5)
    off = _offsets(counts)
    av, wgv = _values(*(t.cuda() for t in (a, sa, wg, sg)))
    gate, gsize = (t.cpu() for t in _product(av, wgv, off))
    up, usize = (t.cpu() for t in _product(av, _values(*(t.cuda() for t in (a, sa, wu, su)))[1], off))
    h = gate * torch.sigmoid(gate) * up
    nb = (n + 127) // 128
    ws = torch.full((moe.moe_query_block_swiglu(rows, n, k, groups),), 0xff, dtype=torch.uint8, device="cuda")
    res = []
    for with_h in (True, False):
        hq = torch.full((rows + 1, n), 77, dtype=torch.uint8, device="cuda")
        hs = torch.full((nb * rows + 1,), 77.0, device="cuda")
        hb = torch.full((rows + 1, n), 77, dtype=torch.bfloat16, device="cuda")
        moe.moe_block_gemm_swiglu(u8(a), sa.cuda(), u8(wg), sg.cuda(), u8(wu), su.cuda(), hq[:-1],
                                  hs[:-1].view(nb, rows), ws, h=hb[:-1] if with_h else None, offsets=off.cuda())
        torch.cuda.synchronize()
        res.append((hq.cpu(), hs.cpu(), hb.cpu()))
    (hq, hs, hb), (hq2, hs2, _) = res
    assert torch.equal(hq, hq2) and torch.equal(hs, hs2)
    hs = hs[:-1].view(nb, rows)
    assert (hq[m:] == 77).all() and (hs[:, m:] == 77).all() and (hb[m:] == 77).all()
    if not m:
        return
    # |silu'| <= 1.1 and |silu(g)| <= |g|: how far h may be off in fp32 (its own few roundings in the 2^-18)
    dg, du = gsize[:m] * CUT, usize[:m] * CUT
    tol = 1.1 * dg * (up[:m].abs() + du) + gate[:m].abs() * du + h[:m].abs() * 2.0 ** -18
    assert ((hb[:m].double() - h[:m]).abs() <= (h[:m].abs() + tol) * HALF + tol).all()
    # h in bf16 and the codes are two roundings of one fp32 value: the code's value is within half a step of
    # E4M3 (2^-4 of it, or 2^-10 scales below the normal codes) and half a step of bf16 of the bf16 one
    s = hs.double().t().repeat_interleave(128, 1)[:m, :n]
    held = hq[:m].view(torch.float8_e4m3fn).double() * s
    near = hb[:m].double()
    assert ((held - near).abs() <= near.abs() * (2.0 ** -4 + HALF) * 1.01 + s * 2.0 ** -10).all()
    for b in range(nb):  # the scale: a power of two, the smallest that the block fits (up to bf16's rounding)
        amax = near[:, 128 * b:128 * b + 128].abs().amax(1)
        assert (torch.frexp(hs[b, :m])[0] == 0.5).all()
        assert (amax <= 448 * hs[b, :m].double() * (1 + HALF)).all()
        assert ((amax >= 224 * hs[b, :m].double() * (1 - HALF)) | (hs[b, :m] <= 2.0 ** -126)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n,k,groups", [(1024, 2048, 6), (144, 656, 20)])
def test_swiglu_workspace_of_the_largest_batch(gpu_lib, n, k, groups):
    """Batches of 12000 rows and fewer, in tiles and in the few-row form, in one workspace sized for the largest:
    the bits that each gives in its own, and nothing behind it."""
    g = torch.Generator(device="cuda").manual_seed(n)
    draw = lambda *shape: torch.randint(-2, 3, shape, generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    wg, wu = draw(groups, n, k), draw(groups, n, k)
    sw = torch.full((groups, (n + 127) // 128, (k + 127) // 128), 2.0 ** -8, device="cuda")
    need = moe.moe_query_block_swiglu(12000, n, k, groups)
    ws = torch.full((need + 64,), 77, dtype=torch.uint8, device="cuda")
    for rows in (12000, 3000, 700, 64, 6, 1):
        counts = _uneven(rows, groups)
        rows = sum(counts) or 1
        a, sa = draw(rows, k), torch.ones((k + 127) // 128, rows, device="cuda")
        off = _offsets(counts if sum(counts) else [1] + [0] * (groups - 1)).cuda()
        res = []
        for buf in (ws[:need], torch.empty(moe.moe_query_block_swiglu(rows, n, k, groups), dtype=torch.uint8, device="cuda")):
            hq, hs = torch.empty(rows, n, dtype=torch.uint8, device="cuda"), torch.empty((n + 127) // 128, rows, device="cuda")
            moe.moe_block_gemm_swiglu(a, sa, wg, sw, wu, sw, hq, hs, buf, offsets=off)
            res.append((hq, hs))
        assert all(torch.equal(x, y) for x, y in zip(*res))
        assert (ws[need:] == 77).all()


@pytest.mark.gpu
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("counts", [[1, 0, 2, 1] * 10, [0, 16, 3, 37, 8] * 8, [25, 20, 30, 40, 0] * 8, [2, 0, 1] * 200], ids=_name)
def test_weights_past_the_last_cache(gpu_lib, counts, glu):
    """More than 2^28 bytes of weights for few rows to a group, in every form they fall to: whole numbers, exact sums."""
    groups, spare = len(counts), 2
    n, k = (2064, 3600) if groups < 100 else (528, 1168)
    n = n if glu else 2 * n + 8
    rows = sum(counts) + spare
    g = torch.Generator(device="cuda").manual_seed(groups + rows)
    draw = lambda *shape: torch.randint(-2, 3, shape, generator=g, device="cuda").to(torch.float8_e4m3fn)
    a, ws = draw(rows, k), [draw(groups, n, k) for _ in range(2 if glu else 1)]
    sa = torch.exp2(torch.randint(-2, 3, ((k + 127) // 128, rows), generator=g, device="cuda").float())
    sw = torch.exp2(torch.randint(-8, -6, (groups, (n + 127) // 128, (k + 127) // 128), generator=g, device="cuda").float())
    off = _offsets(counts)
    want = []
    for w in ws:
        want.append(torch.full((rows, n), float("nan"), dtype=torch.float64, device="cuda"))
        for e in range(groups):
            lo, hi = off[e].item(), off[e + 1].item()
            if hi > lo:
                av, wv = _values(a[lo:hi], sa[:, lo:hi], w[e:e + 1], sw[e:e + 1])
                want[-1][lo:hi] = av @ wv[0].t()
    m, u = sum(counts), lambda t: t.view(torch.uint8)
    out = torch.full((rows, n), 77, dtype=torch.bfloat16, device="cuda")
    if not glu:
        moe.moe_block_gemm(u(a), sa, u(ws[0]), sw, out, offsets=off.cuda())
        assert torch.equal(out[:m], want[0][:m].float().bfloat16()) and (out[m:] == 77).all()
        return
    nb = (n + 127) // 128
    hq, hs = torch.full((rows, n), 77, dtype=torch.uint8, device="cuda"), torch.full((nb, rows), 77.0, device="cuda")
    buf = torch.empty(moe.moe_query_block_swiglu(rows, n, k, groups), dtype=torch.uint8, device="cuda")
    moe.moe_block_gemm_swiglu(u(a), sa, u(ws[0]), sw, u(ws[1]), sw, hq, hs, buf, h=out, offsets=off.cuda())
    h = (want[0] * torch.sigmoid(want[0]) * want[1])[:m]
    near = out[:m].double()
    # (a hardware exponential and reciprocal of a few 2^-24 of the value each, in front of the rounding)
    assert ((near - h).abs() <= h.abs() * HALF * 1.01 + h.abs() * 2.0 ** -18).all()
    s = hs.double().t().repeat_interleave(128, 1)[:m, :n]
    held = hq[:m].view(torch.float8_e4m3fn).double() * s
    assert ((held - near).abs() <= near.abs() * (2.0 ** -4 + HALF) * 1.01 + s * 2.0 ** -10).all()
    assert (out[m:] == 77).all() and (hq[m:] == 77).all() and (hs[:, m:] == 77).all()


@pytest.mark.gpu
def test_codes_in_torch_s_own_type(gpu_lib):
    """Every call takes torch.float8_e4m3fn where it takes bytes, and gives the same bits; other 8-bit types are refused."""
    g = torch.Generator(device="cuda").manual_seed(21)
    T, k, H, I, E = 20, 2, 272, 144, 3
    R, f8 = T * k, torch.float8_e4m3fn
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    W = [torch.randn(E, *s, generator=g, device="cuda").mul(0.1).bfloat16() for s in ((H, I), (H, I), (I, H))]
    at = torch.randperm(R, generator=g, device="cuda").view(T, k).int()
    off, topk_w = _offsets([13, 0, 27]).cuda(), torch.rand(T, k, generator=g, device="cuda")
    new = lambda dtype, *shape: torch.zeros(*shape, dtype=torch.uint8, device="cuda").view(dtype)
    scales = lambda *shape: torch.zeros(shape, device="cuda")
    ws = torch.empty(moe.moe_query_block_swiglu(R, I, H, E), dtype=torch.uint8, device="cuda")

    def layer(dtype):
        xq, xs, hq, hs = new(dtype, R, H), scales(3, R), new(dtype, R, I), scales(2, R)
        w = []
        for v in W:
            kk, n = v.shape[1:]
            w += [new(dtype, E, n, kk), scales(E, (n + 127) // 128, (kk + 127) // 128)]
            moe.moe_block_quantize_weights(v, w[-2], w[-1], transposed=True)
        moe.moe_dispatch_rows(x, at, codes=xq, scales=xs)
        moe.moe_block_gemm_swiglu(xq, xs, *w[:4], hq, hs, ws, offsets=off)
        y, held, back = (torch.zeros(R, n, dtype=torch.bfloat16, device="cuda") for n in (H, I, H))
        moe.moe_block_gemm(hq, hs, *w[4:], y, offsets=off)
        moe.moe_block_dequantize(hq, hs, held)
        dq, ds, bq, bs = new(dtype, R, H), scales(3, R), new(dtype, R, H), scales(3, R)
        moe.moe_block_quantize(y, dq, ds)
        moe.moe_combine_rows_bwd(x, at, topk_w=topk_w, codes=bq, scales=bs)
        wv = torch.zeros(E, H, I, dtype=torch.bfloat16, device="cuda")
        moe.moe_block_dequantize(*w[4:], wv, weights=True)
        return [t.view(torch.uint8) for t in (xq, xs, hq, hs, *w, y, held, dq, ds, bq, bs, wv)]

    assert all(torch.equal(a, b) for a, b in zip(layer(torch.uint8), layer(f8)))
    for other in (torch.int8, torch.float8_e5m2, torch.float8_e4m3fnuz):
        with pytest.raises(moe.MoeError) as e:
            layer(other)
        assert e.value.status == moe.MOE_E_INVALID


@pytest.mark.gpu
def test_turned_weights_give_the_input_gradient(gpu_lib):
    """dA = dOut W: the product with the same blocks turned, against the formula and against a difference."""
    g = torch.Generator().manual_seed(3)
    E, K, N, counts = 3, 272, 144, [20, 0, 41]
    W = torch.randint(-2, 3, (E, K, N), generator=g).bfloat16()  # [E, in, out], as moe_prepare_weights takes it
    rows, off = sum(counts), _offsets(counts).cuda()
    blocks = lambda x: (x + 127) // 128
    fw, fs = torch.empty(E, N, K, dtype=torch.uint8, device="cuda"), torch.empty(E, blocks(N), blocks(K), device="cuda")
    bw, bs = torch.empty(E, K, N, dtype=torch.uint8, device="cuda"), torch.empty(E, blocks(K), blocks(N), device="cuda")
    moe.moe_block_quantize_weights(W.cuda(), fw, fs, transposed=True)
    moe.moe_block_quantize_weights(W.cuda(), bw, bs)
    assert torch.equal(bs, fs.transpose(1, 2)) and torch.equal(bw, fw.transpose(1, 2))

    def product(v, w, s, n):
        q, sc = torch.empty(v.shape, dtype=torch.uint8, device="cuda"), torch.empty(blocks(v.shape[1]), rows, device="cuda")
        moe.moe_block_quantize(v.cuda(), q, sc)
        out = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
        moe.moe_block_gemm(q, sc, w, s, out, offsets=off)
        return out.cpu().double()

    dout = torch.randint(-1, 2, (rows, N), generator=g).bfloat16()
    a = torch.randint(-2, 3, (rows, K), generator=g).bfloat16()
    da = product(dout, bw, bs, K)
    grp = torch.repeat_interleave(torch.arange(E), torch.tensor(counts))
    want = torch.stack([W[grp[r]].double() @ dout[r].double() for r in range(rows)])
    assert torch.equal(da, want.float().bfloat16().double())
    exact = lambda v: torch.stack([v[r].double() @ W[grp[r]].double() for r in range(rows)])
    assert torch.equal(product(a, fw, fs, N), exact(a).float().bfloat16().double())
    for r, c in ((0, 0), (rows - 1, K - 1), (25, 130)):
        a2 = a.clone()
        a2[r, c] += 1
        d = ((exact(a2) - exact(a)) * dout.double()).sum()
        assert d.float().bfloat16().double() == da[r, c]


@pytest.mark.gpu
def test_product_nan_codes_and_offsets_outside(gpu_lib):
    g = torch.Generator().manual_seed(4)
    rows, n, k = 40, 136, 400
    a, sa, w, sw = _operands(g, rows, k, 2, n, True)
    off = _offsets([25, 15])
    ref = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    moe.moe_block_gemm(u8(a), sa.cuda(), u8(w), sw.cuda(), ref, offsets=off.cuda())
    a2, w2 = a.view(torch.uint8).clone(), w.view(torch.uint8).clone()
    a2[7, 399] = 0x7f    # the last value of a row whose last block is short: the next row is sound
    w2[1, 3, 5] = 0xff
    out = torch.empty_like(ref)
    moe.moe_block_gemm(a2.cuda(), sa.cuda(), w2.cuda(), sw.cuda(), out, offsets=off.cuda())
    bad = torch.zeros(rows, n, dtype=torch.bool)
    bad[7], bad[25:, 3] = True, True
    assert torch.isnan(out.cpu()[bad]).all() and torch.equal(out.cpu()[~bad], ref.cpu()[~bad])
    # bounds outside the rows are cut off; the error report of moe_dispatch_layout names no row of the last group
    for bounds, live in (([-5, 25, 99], [(0, 25, 0), (25, 40, 1)]), ([0, 25, -1], [(0, 25, 0)]),
                         ([0, 1 << 30, 1 << 30], [(0, 40, 0)]), ([50, 60, 70], [])):
        out = torch.full((rows + 1, n), 77, dtype=torch.bfloat16, device="cuda")
        moe.moe_block_gemm(u8(a), sa.cuda(), u8(w), sw.cuda(), out[:-1],
                           offsets=torch.tensor(bounds, dtype=torch.int32, device="cuda"))
        want = torch.full((rows + 1, n), 77.0, dtype=torch.float64)
        av, wv = _values(a, sa, w, sw)
        for lo, hi, e in live:
            want[lo:hi] = av[lo:hi] @ wv[e].t()
        assert torch.equal(out.cpu(), want.float().bfloat16())


# rows, groups, n, k that fall to the few-row form and to each of the tiles (of the plain product, and with SwiGLU)
FORMS = [(60, 2, 144, 400), (4100, 40, 1040, 656), (12000, 3, 4112, 272), (1500, 40, 1040, 144), (2300, 40, 272, 656),
         (700, 40, 1040, 656), (300, 40, 4112, 272), (1300, 600, 144, 272)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,groups,n,k", FORMS)
def test_nan_codes_reach_their_own_outputs_only(gpu_lib, rows, groups, n, k):
    g = torch.Generator().manual_seed(rows + n)
    counts = _uneven(rows, groups)
    rows = sum(counts)
    a, sa, w, sw = _operands(g, rows, k, groups, n, True)
    sw = sw * 2.0 ** -8
    off = _offsets(counts)
    e = max(range(groups), key=lambda i: counts[i])  # the group whose matrix is spoilt
    lo, hi = off[e].item(), off[e + 1].item()
    r0 = 0 if e else hi if hi < rows else 0
    r0 = r0 if not lo <= r0 < hi else rows - 1
    a2, w2 = a.view(torch.uint8).clone(), w.view(torch.uint8).clone()
    a2[r0, k - 1], w2[e, n - 5, 5] = 0x7f, 0xff
    bad = torch.zeros(rows, n, dtype=torch.bool, device="cuda")
    bad[r0], bad[lo:hi, n - 5] = True, True
    sa, sw, off = sa.cuda(), sw.cuda(), off.cuda()
    outs = []
    for ac, wc in ((u8(a), u8(w)), (a2.cuda(), w2.cuda())):
        out = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
        moe.moe_block_gemm(ac, sa, wc, sw, out, offsets=off)
        ws = torch.empty(moe.moe_query_block_swiglu(rows, n, k, groups), dtype=torch.uint8, device="cuda")
        hq, hs = torch.empty(rows, n, dtype=torch.uint8, device="cuda"), torch.empty((n + 127) // 128, rows, device="cuda")
        h = torch.empty_like(out)
        moe.moe_block_gemm_swiglu(ac, sa, u8(w), sw, wc, sw, hq, hs, ws, h=h, offsets=off)
        outs.append((out, h, hq.view(torch.float8_e4m3fn).float(), hs))
    (out, h, hq, hs), (out2, h2, hq2, hs2) = outs
    for x, y in ((out, out2), (h, h2)):
        assert torch.isnan(y[bad]).all() and torch.equal(x[~bad], y[~bad])
    assert torch.isnan(hq2[bad]).all() and not torch.isnan(hq2[~bad]).any()
    # the block's scale comes from the other values: it differs where the spoilt one was the largest
    same = (hs == hs2).t().repeat_interleave(128, 1)[:, :n] & ~bad
    assert torch.equal(hq[same], hq2[same]) and same[~bad].float().mean() > 0.9


@pytest.mark.gpu
@pytest.mark.parametrize("rows,groups,n,k", FORMS)
def test_a_captured_graph_follows_new_offsets(gpu_lib, rows, groups, n, k):
    """Both products captured once and replayed on other tables, operands and scales in the same buffers."""
    g = torch.Generator().manual_seed(rows + n + 1)
    counts = _uneven(rows, groups)
    rows = sum(counts)
    sets = []
    for i in range(3):
        a, sa, w, sw = _operands(g, rows, k, groups, n)
        turned = counts[i % groups:] + counts[:i % groups]
        if i == 2:
            turned[0] = 0  # fewer rows than the buffers hold
        sets.append((u8(a), sa.cuda(), u8(w), sw.cuda() * 1e-4, _offsets(turned).cuda()))
    bufs = [t.clone() for t in sets[0]]
    a, sa, w, sw, off = bufs
    out = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    hq, hs = torch.empty(rows, n, dtype=torch.uint8, device="cuda"), torch.empty((n + 127) // 128, rows, device="cuda")
    h, ws = torch.empty_like(out), torch.empty(moe.moe_query_block_swiglu(rows, n, k, groups), dtype=torch.uint8, device="cuda")

    def step():
        moe.moe_block_gemm(a, sa, w, sw, out, offsets=off)
        moe.moe_block_gemm_swiglu(a, sa, w, sw, w, sw, hq, hs, ws, h=h, offsets=off)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for new in sets + sets[:1]:
        for t, v in zip(bufs, new):
            t.copy_(v)
        res = []
        for run in (step, graph.replay):
            for t in (out, hq, hs, h, ws):
                t.fill_(7)
            run()
            torch.cuda.synchronize()
            res.append([t.clone() for t in (out, hq, hs, h)])
        assert all(torch.equal(x, y) for x, y in zip(*res))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,groups,n,k", FORMS)
def test_extreme_scales_in_every_form(gpu_lib, rows, groups, n, k):
    """Row scales of 2^100 and 2^-100 in turn; their products with the weights' go down to 2^-126, the smallest normal
    number, and up to 2^110, at which no sum of whole numbers below 2^13 overflows: exact sums."""
    g = torch.Generator().manual_seed(rows + n + 2)
    counts = _uneven(rows, groups)
    rows = sum(counts)
    a, sa, w, sw = _operands(g, rows, k, groups, n, True)
    off = _offsets(counts)
    sa = torch.exp2(torch.tensor([100.0, -100.0])[torch.arange(rows) % 2]).expand_as(sa).contiguous()
    for scale in (2.0 ** -26, 2.0 ** 10, 1.0):
        sw = torch.full_like(sw, scale)
        want, _ = _product(*_values(a.cuda(), sa.cuda(), w.cuda(), sw.cuda()), off)
        out = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
        moe.moe_block_gemm(u8(a), sa.cuda(), u8(w), sw.cuda(), out, offsets=off.cuda())
        assert torch.equal(out, want.float().bfloat16())


BOUNDS = [([-5, 25, 40, 1 << 20], [(0, 25, 0), (25, 40, 1), (40, None, 2)]), ([0, 25, 30, -1], [(0, 25, 0), (25, 30, 1)]),
          ([0, 1 << 30, 1 << 30, -1], [(0, None, 0)]), ([50000, 60000, 70000, 80000], []), ([0, 0, 0, -1], []),
          ([7, 7, 30, 30], [(7, 30, 1)])]


@pytest.mark.gpu
@pytest.mark.parametrize("n,k,rows", [(144, 400, 60), (272, 144, 50), (1040, 528, 3000), (528, 656, 1200), (2064, 272, 9000)])
@pytest.mark.parametrize("glu", [False, True])
def test_bounds_outside_the_rows(gpu_lib, n, k, rows, glu):
    """In the few-row form and in tiles: bounds are cut off, a last one of -1 names no row, other rows are left."""
    g = torch.Generator().manual_seed(n + rows)
    a, sa, w, sw = _operands(g, rows, k, 3, n, True)
    sw = sw * 2.0 ** -8
    a, sa, w, sw = a.cuda(), sa.cuda(), w.cuda(), sw.cuda()
    av, wv = _values(a, sa, w, sw)
    byte = lambda t: t.view(torch.uint8)
    nb = (n + 127) // 128
    ws = torch.empty(moe.moe_query_block_swiglu(rows, n, k, 3), dtype=torch.uint8, device="cuda") if glu else None
    for bounds, live in BOUNDS:
        off = torch.tensor(bounds, dtype=torch.int32, device="cuda")
        out = torch.full((rows + 1, n), 77, dtype=torch.bfloat16, device="cuda")
        want = torch.full((rows + 1, n), 77.0, dtype=torch.float64, device="cuda")
        named = torch.zeros(rows, dtype=torch.bool, device="cuda")
        for lo, hi, e in live:
            hi = rows if hi is None else hi
            want[lo:hi], named[lo:hi] = av[lo:hi] @ wv[e].t(), True
        if not glu:
            moe.moe_block_gemm(byte(a), sa, byte(w), sw, out[:-1], offsets=off)
            assert torch.equal(out, want.float().bfloat16()), bounds
            continue
        hq = torch.full((rows, n), 77, dtype=torch.uint8, device="cuda")
        hs = torch.full((nb, rows), 77.0, device="cuda")
        moe.moe_block_gemm_swiglu(byte(a), sa, byte(w), sw, byte(w), sw, hq, hs, ws, h=out[:-1], offsets=off)
        h = (want * want * torch.sigmoid(want))[:-1][named]
        near = out[:-1][named].double()
        # (a hardware exponential and reciprocal of a few 2^-24 of the value each, in front of the rounding)
        assert ((near - h).abs() <= h.abs() * HALF * 1.01 + h.abs() * 2.0 ** -18).all(), bounds
        s = hs.double().t().repeat_interleave(128, 1)[:, :n][named]
        held = hq.view(torch.float8_e4m3fn).double()[named] * s
        assert ((held - near).abs() <= near.abs() * (2.0 ** -4 + HALF) * 1.01 + s * 2.0 ** -10).all(), bounds
        assert (out[:-1][~named] == 77).all() and (out[-1] == 77).all() and (hq[~named] == 77).all()
        assert (hs[:, ~named] == 77).all()


@pytest.mark.gpu
@pytest.mark.parametrize("groups,n,k,rows", [(5, 144, 400, 60), (40, 1032, 400, 4100), (40, 528, 656, 7000), (3, 2064, 272, 9000),
                                             (600, 136, 272, 1300), (16384, 8, 16, 1 << 24)])
def test_a_table_of_anything(gpu_lib, groups, n, k, rows):
    """moe_dispatch_layout leaves the table unwritten where it reports an error, and the calls behind it are under
    way by then: they end, and write nothing outside their outputs.  (The last case: groups of all rows would make
    2^31 parts.)"""
    g = torch.Generator(device="cuda").manual_seed(groups)
    draw = lambda *shape: torch.randint(0, 120, shape, generator=g, device="cuda", dtype=torch.uint8)
    scales = lambda *shape: torch.ones(shape, device="cuda")
    a, sa, w = draw(rows, k), scales((k + 127) // 128, rows), draw(groups, n, k)
    sw = scales(groups, (n + 127) // 128, (k + 127) // 128)
    buf = torch.full((rows + 512, n), 77, dtype=torch.bfloat16, device="cuda")
    tables = [torch.randint(-(1 << 31), 1 << 31, (groups + 1,), generator=g, device="cuda").int(),
              torch.randint(0, rows + 1, (groups + 1,), generator=g, device="cuda").int(),
              (torch.arange(groups + 1, device="cuda") % 2 * rows).int(),
              torch.arange(groups, -1, -1, device="cuda").mul(rows // groups).int()]
    for off in tables:
        print("table %s ..." % off[:4].tolist(), flush=True)
        moe.moe_block_gemm(a, sa, w, sw, buf[256:-256], offsets=off)
        torch.cuda.synchronize()
        assert (buf[:256] == 77).all() and (buf[-256:] == 77).all()
        if n % 16:
            continue
        nb = (n + 127) // 128
        ws = torch.empty(moe.moe_query_block_swiglu(rows, n, k, groups), dtype=torch.uint8, device="cuda")
        hq = torch.full((rows + 512, n), 77, dtype=torch.uint8, device="cuda")
        hs = torch.full((nb * rows + 512,), 77.0, device="cuda")
        moe.moe_block_gemm_swiglu(a, sa, w, sw, w, sw, hq[256:-256], hs[256:-256].view(nb, rows), ws,
                                  h=buf[256:-256], offsets=off)
        torch.cuda.synchronize()
        for t in (buf, hq, hs):
            assert (t[:256] == 77).all() and (t[-256:] == 77).all()


@pytest.mark.gpu
def test_extreme_scales(gpu_lib):
    """Scales far apart whose products are normal numbers, and a result that overflows."""
    a = torch.full((2, 256), 448.0).to(torch.float8_e4m3fn)
    w = torch.full((1, 8, 256), 1.0).to(torch.float8_e4m3fn)
    sa = torch.tensor([[2.0 ** 100, 2.0 ** -100], [2.0 ** 100, 2.0 ** -100]])
    for sw, want in ((2.0 ** -100, [448.0 * 256, 0.0]), (2.0 ** 20, [float("inf"), 448.0 * 256 * 2.0 ** -80]),
                     (2.0 ** -20, [448.0 * 256 * 2.0 ** 80, 448.0 * 256 * 2.0 ** -120])):
        out = torch.empty(2, 8, dtype=torch.bfloat16, device="cuda")
        moe.moe_block_gemm(u8(a), sa.cuda(), u8(w), torch.full((1, 1, 2), sw).cuda(), out)
        for r in range(2):
            if want[r]:
                assert (out[r].double().cpu() == torch.tensor(want[r]).bfloat16().double()).all()


@pytest.mark.gpu
def test_weights_past_32_bits(gpu_lib):
    """Groups whose codes start past 2^32 bytes."""
    E, n, k = 33, 8192, 16384
    w = torch.zeros(E, n, k, dtype=torch.uint8, device="cuda")
    one = int(torch.tensor([1.0]).to(torch.float8_e4m3fn).view(torch.uint8))
    w[32] = one
    sw, sa = torch.ones(E, n // 128, k // 128, device="cuda"), torch.ones(k // 128, 40, device="cuda")
    a = torch.full((40, k), one, dtype=torch.uint8, device="cuda")
    out = torch.empty(40, n, dtype=torch.bfloat16, device="cuda")
    moe.moe_block_gemm(a, sa, w, sw, out, offsets=_offsets([1] * 31 + [0, 9]).cuda())
    assert not out[:31].any() and (out[31:40] == k).all()


@pytest.mark.gpu
def test_captured_and_on_another_stream(gpu_lib):
    g = torch.Generator().manual_seed(12)
    counts, n, k = [3, 0, 70, 300], 256, 384
    rows = sum(counts)
    a, sa, w, sw = _operands(g, rows, k, 4, n)
    a, sa, w, sw, off = u8(a), sa.cuda(), u8(w), sw.cuda() * 1e-4, _offsets(counts).cuda()
    out = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    hq, hs = torch.empty(rows, n, dtype=torch.uint8, device="cuda"), torch.empty(2, rows, device="cuda")
    ws = torch.empty(moe.moe_query_block_swiglu(rows, n, k, 4), dtype=torch.uint8, device="cuda")

    def step():
        moe.moe_block_gemm(a, sa, w, sw, out, offsets=off)
        moe.moe_block_gemm_swiglu(a, sa, w, sw, w, sw, hq, hs, ws, offsets=off)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (out, hq, hs)]
    s = torch.cuda.Stream()
    for t in (out, hq, hs):
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((out, hq, hs), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (out, hq, hs, ws):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((out, hq, hs), want))


@pytest.mark.gpu
def test_two_calls_at_once(gpu_lib):
    """Products of both kinds on two streams, a workspace each, while the other's run: as alone."""
    g = torch.Generator().manual_seed(31)
    jobs = []
    for rows, groups, n, k in ((3000, 5, 1040, 528), (90, 12, 528, 1040)):
        counts = _uneven(rows, groups)
        rows = sum(counts)
        a, sa, wg, sg = _operands(g, rows, k, groups, n)
        _, _, wu, su = _operands(g, 1, k, groups, n)
        off = _offsets(counts).cuda()
        a, wg, wu, sa, sg, su = u8(a), u8(wg), u8(wu), sa.cuda(), sg.cuda() / 1e5, su.cuda() / 1e5
        out = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
        hq, hs = torch.empty(rows, n, dtype=torch.uint8, device="cuda"), torch.empty((n + 127) // 128, rows, device="cuda")
        ws = torch.empty(moe.moe_query_block_swiglu(rows, n, k, groups), dtype=torch.uint8, device="cuda")

        def run(stream, a=a, sa=sa, wg=wg, sg=sg, wu=wu, su=su, out=out, hq=hq, hs=hs, ws=ws, off=off):
            moe.moe_block_gemm(a, sa, wg, sg, out, offsets=off, stream=stream)
            moe.moe_block_gemm_swiglu(a, sa, wg, sg, wu, su, hq, hs, ws, offsets=off, stream=stream)

        run(torch.cuda.current_stream())
        torch.cuda.synchronize()
        jobs.append((run, (out, hq, hs), [t.clone() for t in (out, hq, hs)], torch.cuda.Stream()))
    for _, outs, _, _ in jobs:
        for t in outs:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for run, _, _, stream in jobs:
            run(stream)
    torch.cuda.synchronize()
    for _, outs, alone, _ in jobs:
        assert all(torch.equal(x, y) for x, y in zip(outs, alone))


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I,E,k", [(1, 128, 64, 8, 2), (9, 256, 144, 5, 3), (200, 384, 256, 4, 2)])
def test_the_layer_in_parts(gpu_lib, T, H, I, E, k):
    """Router, layout, rows of codes, both products and the weighted sum in a row, as a server runs them,
    against the layer's formula in 64 bits on the values that the codes stand for."""
    g = torch.Generator().manual_seed(T + H)
    dev = lambda t: t.cuda()
    x = torch.randn(T, H, generator=g).bfloat16()
    Wr = torch.randn(H, E, generator=g) * 0.05
    Wg, Wu, Wd = (torch.randn(E, *s, generator=g).mul(0.05).bfloat16() for s in ((H, I), (H, I), (I, H)))
    cfg = moe.make_cfg(T, (H + 63) // 64 * 64, 64, E, k)
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, counts, offsets, row_token, tok_row = (torch.empty(s, **i32) for s in ((T, k), E, E + 1, T * k, (T, k)))
    topk_w = torch.empty(T, k, device="cuda")
    moe.moe_route(cfg, dev(x), dev(Wr), None, idx, topk_w)
    moe.moe_dispatch_layout(cfg, idx, counts, offsets, row_token, tok_row)
    packed = []
    for W in (Wg, Wu, Wd):
        n, kk = W.shape[2], W.shape[1]
        q, s = torch.empty(E, n, kk, dtype=torch.uint8, device="cuda"), torch.empty(E, (n + 127) // 128, (kk + 127) // 128, device="cuda")
        moe.moe_block_quantize_weights(dev(W), q, s, transposed=True)
        v = torch.empty(E, n, kk, dtype=torch.bfloat16, device="cuda")
        moe.moe_block_dequantize(q, s, v, weights=True)
        packed.append((q, s, v.cpu().double()))
    R = T * k
    codes = lambda rows, cols: (torch.empty(rows, cols, dtype=torch.uint8, device="cuda"),
                                torch.empty((cols + 127) // 128, rows, device="cuda"))
    xq, xs = codes(R, H)
    hq, hs = codes(R, I)
    y, out = torch.empty(R, H, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_query_block_swiglu(R, I, H, E), dtype=torch.uint8, device="cuda")
    (gq, gs, gv), (uq, us, uv), (dq, ds, dv) = packed
    moe.moe_dispatch_rows(dev(x), tok_row, codes=xq, scales=xs)
    moe.moe_block_gemm_swiglu(xq, xs, gq, gs, uq, us, hq, hs, ws, offsets=offsets)
    moe.moe_block_gemm(hq, hs, dq, ds, y, offsets=offsets)
    moe.moe_combine_rows(y, tok_row, out, topk_w=topk_w)
    torch.cuda.synchronize()
    qx, sx = _row_codes(x.double().numpy())
    xv = torch.from_numpy(qx).view(torch.float8_e4m3fn).double() * torch.from_numpy(sx).double().t().repeat_interleave(128, 1)[:, :H]
    want = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = idx[t, j].item()
            gate = gv[e] @ xv[t]
            h = gate * torch.sigmoid(gate) * (uv[e] @ xv[t])
            want[t] += topk_w[t, j].item() * (dv[e] @ h)
    # h is held in 8 bits (2^-4 of a value at most, a third of that in the mean) and enters a sum of I terms:
    # against the unquantised h the output is off by about 2^-5.5 of its own size, at most
    assert (out.cpu().double() - want).norm() <= want.norm() * 2.0 ** -4.5


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I,E,k", [(1, 128, 64, 8, 2), (9, 256, 144, 5, 3), (200, 384, 256, 4, 2), (2000, 512, 528, 6, 3)])
def test_the_layer_in_parts_call_by_call(gpu_lib, T, H, I, E, k):
    """The same run, each call against the formula in 64 bits on what the call before it gave: the codes of h that the
    down product takes, its rows that the sum takes.  So no step's own quantisation stands in the next one's bound."""
    g = torch.Generator(device="cuda").manual_seed(T + H)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    packed = []
    for n, kk in ((I, H), (I, H), (H, I)):
        q, s = torch.empty(E, n, kk, dtype=torch.uint8, device="cuda"), torch.empty(E, (n + 127) // 128, (kk + 127) // 128, device="cuda")
        moe.moe_block_quantize_weights(torch.randn(E, kk, n, generator=g, device="cuda").mul(0.05).bfloat16(), q, s, transposed=True)
        packed.append((q, s))
    cfg = moe.make_cfg(T, (H + 63) // 64 * 64, 64, E, k)
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, counts, offsets, row_token, tok_row = (torch.empty(s, **i32) for s in ((T, k), E, E + 1, T * k, (T, k)))
    topk_w = torch.empty(T, k, device="cuda")
    moe.moe_route(cfg, x, torch.randn(H, E, generator=g, device="cuda") * 0.05, None, idx, topk_w)
    moe.moe_dispatch_layout(cfg, idx, counts, offsets, row_token, tok_row)
    R = T * k
    codes = lambda rows, cols: (torch.empty(rows, cols, dtype=torch.uint8, device="cuda"),
                                torch.empty((cols + 127) // 128, rows, device="cuda"))
    (xq, xs), (hq, hs) = codes(R, H), codes(R, I)
    y, out = torch.empty(R, H, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    h = torch.empty(R, I, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_query_block_swiglu(R, I, H, E), dtype=torch.uint8, device="cuda")
    moe.moe_dispatch_rows(x, tok_row, codes=xq, scales=xs)
    moe.moe_block_gemm_swiglu(xq, xs, *packed[0], *packed[1], hq, hs, ws, h=h, offsets=offsets)
    moe.moe_block_gemm(hq, hs, *packed[2], y, offsets=offsets)
    moe.moe_combine_rows(y, tok_row, out, topk_w=topk_w)
    torch.cuda.synchronize()
    f8 = lambda t: t.view(torch.float8_e4m3fn)
    off = offsets.cpu()
    # x's codes are one rounding of x each, within half a step of E4M3 (2^-4 of it, 2^-10 of the scale below the normal codes)
    sx = xs.double().t().repeat_interleave(128, 1)[:, :H]
    rows = x[row_token.long()].double()
    assert ((f8(xq).double() * sx - rows).abs() <= rows.abs() * 2.0 ** -4 + sx * 2.0 ** -10).all()
    (gate, gs), (up, us) = (_product(*_values(f8(xq), xs, f8(q), s), off) for q, s in packed[:2])
    hw = gate * torch.sigmoid(gate) * up
    dg, du = gs * CUT, us * CUT
    tol = 1.1 * dg * (up.abs() + du) + gate.abs() * du + hw.abs() * 2.0 ** -18
    assert ((h.double() - hw).abs() <= (hw.abs() + tol) * HALF + tol).all()
    sh = hs.double().t().repeat_interleave(128, 1)[:, :I]
    held, near = f8(hq).double() * sh, h.double()
    assert ((held - near).abs() <= near.abs() * (2.0 ** -4 + HALF) * 1.01 + sh * 2.0 ** -10).all()
    yw, size = _product(*_values(f8(hq), hs, f8(packed[2][0]), packed[2][1]), off)
    assert ((y.double() - yw).abs() <= yw.abs() * HALF + size * CUT * 1.01).all()
    assert (y.double() - yw).norm() <= yw.norm() * HALF * 1.125
    terms = y.double()[tok_row.long()] * topk_w.double()[..., None]
    want, size = terms.sum(1), terms.abs().sum(1)
    assert ((out.double() - want).abs() <= want.abs() * HALF + (k + 1) * 2.0 ** -24 * size * 1.01).all()
