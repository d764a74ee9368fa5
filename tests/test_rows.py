"""Rows by expert and back (moe_dispatch_rows, moe_combine_rows, moe_combine_rows_bwd): refusals on the
CPU, and on the GPU the outputs against 64-bit formulas.

Bounds.  The sum over k choices is k fused multiply-adds in fp32, each off by at most 2^-24 of the sum of
magnitudes, and one rounding to bf16 (2^-8 of the value).  A dot product over cols is at most cols / 8 / 16
+ 8 additions in one lane's chain and ten joins: (cols / 16 + 20) 2^-24 of the sum of magnitudes covers it.
w * dout is one fp32 product and one rounding: 2^-8 + 2^-24 of the value."""
import numpy as np
import pytest
import torch

import dispatch_grouped_gemm_moe_amd as moe

FAKE = 1 << 20
HALF = 2.0 ** -8


# ------------------------------------------------------------------ refusals (no GPU)

def _dispatch(tokens=4, k=2, cols=64, rows=8, **over):
    a = dict(x=FAKE, at=FAKE, dst=FAKE, codes=None, scales=None)
    a.update(over)
    return moe.lib().moe_dispatch_rows(tokens, k, cols, rows, a["x"], a["at"], a["dst"], a["codes"], a["scales"], None)


def _combine(tokens=4, k=2, cols=64, rows=8, **over):
    a = dict(src=FAKE, at=FAKE, w=None, add=None, out=FAKE)
    a.update(over)
    return moe.lib().moe_combine_rows(tokens, k, cols, rows, a["src"], a["at"], a["w"], a["add"], a["out"], None)


def _bwd(tokens=4, k=2, cols=64, rows=8, **over):
    a = dict(dout=FAKE, src=FAKE, at=FAKE, w=None, dsrc=FAKE, codes=None, scales=None, dw=FAKE)
    a.update(over)
    return moe.lib().moe_combine_rows_bwd(tokens, k, cols, rows, a["dout"], a["src"], a["at"], a["w"], a["dsrc"],
                                          a["codes"], a["scales"], a["dw"], None)


SIZES = [dict(tokens=0), dict(tokens=-1), dict(k=0), dict(cols=0), dict(cols=-8), dict(cols=12), dict(rows=0),
         dict(at=None), dict(at=FAKE + 2)]
TOO_BIG = [dict(k=17), dict(cols=(1 << 20) + 16), dict(tokens=(1 << 29) + 1), dict(rows=(1 << 30) + 1)]


@pytest.mark.parametrize("kw", SIZES + [dict(x=None), dict(x=FAKE + 8), dict(dst=None), dict(dst=FAKE + 8),
                                        dict(codes=FAKE), dict(scales=FAKE), dict(codes=FAKE + 8, scales=FAKE),
                                        dict(codes=FAKE, scales=FAKE + 2), dict(cols=24, codes=FAKE, scales=FAKE)])
def test_dispatch_refuses(kw):
    assert _dispatch(**kw) == moe.MOE_E_INVALID


@pytest.mark.parametrize("kw", SIZES + [dict(src=None), dict(out=None), dict(src=FAKE + 8), dict(w=FAKE + 2),
                                        dict(add=FAKE + 8), dict(out=FAKE + 2)])
def test_combine_refuses(kw):
    assert _combine(**kw) == moe.MOE_E_INVALID


@pytest.mark.parametrize("kw", SIZES + [dict(dout=None), dict(src=None), dict(dsrc=None, dw=None),
                                        dict(dout=FAKE + 8), dict(src=FAKE + 8), dict(w=FAKE + 1),
                                        dict(dsrc=FAKE + 8), dict(dw=FAKE + 2), dict(codes=FAKE), dict(scales=FAKE),
                                        dict(codes=FAKE + 4, scales=FAKE), dict(cols=8, codes=FAKE, scales=FAKE)])
def test_combine_backward_refuses(kw):
    assert _bwd(**kw) == moe.MOE_E_INVALID


@pytest.mark.parametrize("kw", TOO_BIG)
def test_sizes_beyond_the_kernels(kw):
    for call in (_dispatch, _combine, _bwd):
        assert call(**kw) == moe.MOE_E_UNSUPPORTED


def test_binding_refuses_tensors_the_kernels_cannot_read():
    b16, i32 = torch.bfloat16, torch.int32
    x, at, rows = torch.zeros(4, 64, dtype=b16), torch.zeros(4, 2, dtype=i32), torch.zeros(8, 64, dtype=b16)
    good = dict(x=x, tok_row=at, dst=rows, stream=0)
    for kw in (dict(), dict(x=x.float()), dict(x=torch.zeros(64, 4, dtype=b16).t()), dict(tok_row=at.long()),
               dict(tok_row=at[:3]), dict(dst=None), dict(codes=torch.zeros(7, 64, dtype=torch.uint8)),
               dict(codes=torch.zeros(8, 64, dtype=torch.uint8), scales=torch.zeros(7)), dict(dst=rows.to("meta")),
               # another number of rows would be another layout of the scales
               dict(codes=torch.zeros(9, 64, dtype=torch.uint8), scales=torch.zeros(1, 9)),
               dict(codes=torch.zeros(8, 64, dtype=torch.uint8), scales=torch.zeros(1, 9))):
        with pytest.raises(moe.MoeError) as e:  # (the first: host tensors)
            moe.moe_dispatch_rows(**{**good, **kw})
        assert e.value.status == moe.MOE_E_INVALID
    good = dict(src=rows, tok_row=at, out=x, stream=0)
    for kw in (dict(), dict(out=x[:3]), dict(topk_w=torch.zeros(4, 2, dtype=b16)), dict(add=x[:, ::2]),
               dict(topk_w=torch.zeros(3, 2))):
        with pytest.raises(moe.MoeError) as e:
            moe.moe_combine_rows(**{**good, **kw})
        assert e.value.status == moe.MOE_E_INVALID
    good = dict(dout=x, tok_row=at, src=rows, dsrc=torch.zeros_like(rows), dw=torch.zeros(4, 2), stream=0)
    for kw in (dict(), dict(dw=torch.zeros(7)), dict(src=rows.float()), dict(dout=x.t().contiguous().t())):
        with pytest.raises(moe.MoeError) as e:
            moe.moe_combine_rows_bwd(**{**good, **kw})
        assert e.value.status == moe.MOE_E_INVALID


# ------------------------------------------------------------------ GPU

def _table(g, T, k, dropped=0.0, spare=0):
    """A table of distinct rows in random order, some choices without one (of several kinds), and its rows."""
    keep = torch.rand(T, k, generator=g) >= dropped
    rows = int(keep.sum()) + spare
    at = torch.full((T, k), -1, dtype=torch.int32)
    at[keep] = torch.randperm(max(rows, 1), generator=g)[:int(keep.sum())].int()
    none = torch.tensor([-1, -(1 << 31), (1 << 31) - 1, max(rows, 1)], dtype=torch.int32)
    at[~keep] = none[torch.randint(0, 4, (int((~keep).sum()),), generator=g)]
    return at, max(rows, 1)


def _rand(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g).to(dtype)


def _guarded(rows, *more, dtype=torch.bfloat16):
    """An output with a guard row behind it, all 77."""
    return torch.full((rows + 1, *more), 77, dtype=dtype, device="cuda")


CASES = [(1, 1, 8, 0.0, 0), (1, 16, 24, 0.0, 0), (5, 3, 1032, 0.3, 2), (130, 8, 128, 0.0, 0), (33, 2, 144, 0.5, 7),
         (17, 16, 2064, 0.2, 1), (64, 6, 2048, 0.0, 0), (9, 5, 7168, 0.1, 0), (3, 4, 40, 1.0, 0), (257, 1, 16, 0.2, 3),
         (40, 7, 520, 0.1, 0), (6, 9, 4112, 0.4, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,H,dropped,spare", CASES)
def test_dispatch(gpu_lib, T, k, H, dropped, spare):
    g = torch.Generator().manual_seed(T * 100 + k)
    at, rows = _table(g, T, k, dropped, spare)
    x = _rand(g, T, H)
    want = torch.full((rows + 1, H), 77, dtype=torch.bfloat16)
    kept = (at >= 0) & (at < rows)
    for t in range(T):
        for j in range(k):
            if kept[t, j]:
                want[at[t, j]] = x[t]
    dst = _guarded(rows, H)
    moe.moe_dispatch_rows(x.cuda(), at.cuda(), dst=dst[:-1])
    torch.cuda.synchronize()
    assert torch.equal(dst.cpu(), want)
    if H % 16:
        return
    # codes of the same rows, with and without the bf16 ones: the quantiser's, and nothing elsewhere
    nb = (H + 127) // 128
    q, s = torch.zeros(T, H, dtype=torch.uint8, device="cuda"), torch.zeros(nb, T, device="cuda")
    moe.moe_block_quantize(x.cuda(), q, s)
    for with_dst in (False, True):
        codes, scales, dst = _guarded(rows, H, dtype=torch.uint8), torch.full((nb, rows), 77.0, device="cuda"), _guarded(rows, H)
        moe.moe_dispatch_rows(x.cuda(), at.cuda(), dst=dst[:-1] if with_dst else None, codes=codes[:-1], scales=scales)
        torch.cuda.synchronize()
        wq, ws = torch.full((rows + 1, H), 77, dtype=torch.uint8), torch.full((nb, rows), 77.0)
        for t, j in kept.nonzero().tolist():
            wq[at[t, j]], ws[:, at[t, j]] = q[t].cpu(), s[:, t].cpu()
        assert torch.equal(codes.cpu(), wq) and torch.equal(scales.cpu(), ws)
        if with_dst:
            assert torch.equal(dst.cpu(), want)


def _combined(src, at, w, add):
    """In 64 bits: the sum, and the sum of its terms' magnitudes."""
    T, k = at.shape
    kept = (at >= 0) & (at < src.shape[0])
    v = torch.where(kept[..., None], src.double()[at.long().clamp(0, src.shape[0] - 1)], 0.0)
    terms = v * torch.where(kept, w.double(), 0.0)[..., None]
    base = torch.zeros(T, src.shape[1], dtype=torch.float64) if add is None else add.double()
    return base + terms.sum(1), base.abs() + terms.abs().sum(1)


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,H,dropped,spare", CASES)
def test_combine(gpu_lib, T, k, H, dropped, spare):
    g = torch.Generator().manual_seed(T * 100 + k + 1)
    at, rows = _table(g, T, k, dropped, spare)
    src, add, w = _rand(g, rows, H), _rand(g, T, H), _rand(g, T, k, dtype=torch.float32)
    w[(at < 0) | (at >= rows)] = float("nan")  # a missing row's weight is not used
    for ww in (None, w):
        for aa in (None, add):
            want, size = _combined(src, at, torch.ones(T, k) if ww is None else ww, aa)
            outs = []
            for _ in range(2):
                out = _guarded(T, H)
                moe.moe_combine_rows(src.cuda(), at.cuda(), out[:-1], topk_w=None if ww is None else ww.cuda(),
                                     add=None if aa is None else aa.cuda())
                torch.cuda.synchronize()
                outs.append(out.cpu())
            assert torch.equal(*outs) and (outs[0][-1] == 77).all()
            assert ((outs[0][:-1].double() - want).abs() <= want.abs() * HALF + (k + 1) * 2.0 ** -24 * size * 1.01).all()
            if aa is not None:  # in place
                buf = aa.cuda()
                moe.moe_combine_rows(src.cuda(), at.cuda(), buf, topk_w=None if ww is None else ww.cuda(), add=buf)
                assert torch.equal(buf.cpu(), outs[0][:-1])


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,H,dropped,spare", CASES)
def test_combine_backward(gpu_lib, T, k, H, dropped, spare):
    g = torch.Generator().manual_seed(T * 100 + k + 2)
    at, rows = _table(g, T, k, dropped, spare)
    src, dout, w = _rand(g, rows, H), _rand(g, T, H), _rand(g, T, k, dtype=torch.float32)
    kept = (at >= 0) & (at < rows)
    v = torch.where(kept[..., None], src.double()[at.long().clamp(0, rows - 1)], 0.0)
    dots = v * dout.double()[:, None]
    want_dw, size = dots.sum(2), dots.abs().sum(2)
    for ww in (None, w):
        want = torch.full((rows + 1, H), 77.0, dtype=torch.float64)
        for t, j in kept.nonzero().tolist():
            want[at[t, j]] = dout[t].double() * (1.0 if ww is None else ww[t, j].double())
        kw = dict(topk_w=None if ww is None else ww.cuda())
        d, dw = _guarded(rows, H), torch.full((T * k + 1,), 77.0, device="cuda")
        moe.moe_combine_rows_bwd(dout.cuda(), at.cuda(), src=src.cuda(), dsrc=d[:-1], dw=dw[:-1].view(T, k), **kw)
        torch.cuda.synchronize()
        assert ((d.cpu().double() - want).abs() <= want.abs() * (HALF + 2.0 ** -24)).all()
        got = dw.cpu()
        assert got[-1] == 77
        assert ((got[:-1].view(T, k).double() - want_dw).abs() <= (H / 16 + 20) * 2.0 ** -24 * size).all()
        # each output alone, and a second run: the same bits
        d2, dw2 = _guarded(rows, H), torch.empty(T, k, device="cuda")
        moe.moe_combine_rows_bwd(dout.cuda(), at.cuda(), dsrc=d2[:-1], **kw)
        moe.moe_combine_rows_bwd(dout.cuda(), at.cuda(), src=src.cuda(), dw=dw2, **kw)
        assert torch.equal(d2, d) and torch.equal(dw2.cpu().view(-1), got[:-1])
        if H % 16 == 0:  # codes of the rounded gradient
            nb = (H + 127) // 128
            q, s = torch.zeros(rows, H, dtype=torch.uint8, device="cuda"), torch.zeros(nb, rows, device="cuda")
            moe.moe_block_quantize(d[:-1].contiguous(), q, s)
            codes, scales = _guarded(rows, H, dtype=torch.uint8), torch.full((nb, rows), 77.0, device="cuda")
            moe.moe_combine_rows_bwd(dout.cuda(), at.cuda(), codes=codes[:-1], scales=scales, **kw)
            named = torch.zeros(rows, dtype=torch.bool)
            named[at[kept].long()] = True
            named = named.cuda()
            assert torch.equal(codes[:-1][named], q[named]) and torch.equal(scales[:, named], s[:, named])
            assert (codes[:-1][~named] == 77).all() and (scales[:, ~named] == 77).all() and (codes[-1] == 77).all()


# Tokens enough to fill the CUs (one workgroup walks a row in several pieces), rows wider than a 1024-thread
# workgroup covers at once, and rows past the last cache's 256 MB: T, k, H, dropped, spare
LARGE = [(2100, 3, 2064, 0.1, 5), (2100, 9, 2064, 0.0, 0), (2500, 3, 4112, 0.2, 0), (2100, 9, 4112, 0.1, 3), (2051, 2, 7168, 0.0, 1),
         (16500, 4, 128, 0.1, 0), (33000, 1, 48, 0.0, 2), (3, 2, 8208, 0.0, 0), (5, 9, 16400, 0.3, 1), (1023, 2, 2064, 0.1, 0),
         (1024, 2, 2064, 0.1, 0), (5000, 6, 8208, 0.1, 0), (10000, 8, 4112, 0.1, 0)]


def _large(T, k, H, dropped, spare, seed):
    g = torch.Generator().manual_seed(seed)
    at, rows = _table(g, T, k, dropped, spare)
    kept = (at >= 0) & (at < rows)
    t_of, j_of = (v.cuda() for v in kept.nonzero(as_tuple=True))
    r_of = at[kept].long().cuda()  # row r_of[i] is that of choice (t_of[i], j_of[i])
    free = torch.ones(rows, dtype=torch.bool, device="cuda")
    free[r_of] = False
    return torch.Generator(device="cuda").manual_seed(seed), at.cuda(), rows, t_of, j_of, r_of, free


def _normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,H,dropped,spare", LARGE)
def test_dispatch_of_many_tokens_and_wide_rows(gpu_lib, T, k, H, dropped, spare):
    g, at, rows, t_of, _, r_of, free = _large(T, k, H, dropped, spare, T + k + H)
    x, nb = _normal(g, T, H), (H + 127) // 128
    dst = _guarded(rows, H)
    moe.moe_dispatch_rows(x, at, dst=dst[:-1])
    assert torch.equal(dst[r_of], x[t_of]) and (dst[:-1][free] == 77).all() and (dst[-1] == 77).all()
    q, s = torch.zeros(T, H, dtype=torch.uint8, device="cuda"), torch.zeros(nb, T, device="cuda")
    moe.moe_block_quantize(x, q, s)
    for with_dst in (False, True):
        codes, scales, dst2 = _guarded(rows, H, dtype=torch.uint8), torch.full((nb, rows), 77.0, device="cuda"), _guarded(rows, H)
        moe.moe_dispatch_rows(x, at, dst=dst2[:-1] if with_dst else None, codes=codes[:-1], scales=scales)
        assert torch.equal(codes[r_of], q[t_of]) and torch.equal(scales[:, r_of], s[:, t_of])
        assert (codes[:-1][free] == 77).all() and (codes[-1] == 77).all() and (scales[:, free] == 77).all()
        assert torch.equal(dst2, dst) if with_dst else (dst2 == 77).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,H,dropped,spare", LARGE)
def test_combine_of_many_tokens_and_wide_rows(gpu_lib, T, k, H, dropped, spare):
    g, at, rows, t_of, j_of, r_of, _ = _large(T, k, H, dropped, spare, T + k + H + 1)
    src, add, w = _normal(g, rows, H), _normal(g, T, H), _normal(g, T, k, dtype=torch.float32)
    for ww, aa in ((None, None), (w, add)):
        out = _guarded(T, H)
        moe.moe_combine_rows(src, at, out[:-1], topk_w=ww, add=aa)
        want = torch.zeros(T, H, dtype=torch.float64, device="cuda") if aa is None else aa.double()
        size = want.abs()
        for j in range(k):
            i = (j_of == j).nonzero()[:, 0]
            term = src[r_of[i]].double() * (1.0 if ww is None else ww[t_of[i], j, None].double())
            want[t_of[i]] += term
            size[t_of[i]] += term.abs()
        assert ((out[:-1].double() - want).abs() <= want.abs() * HALF + (k + 1) * 2.0 ** -24 * size * 1.01).all()
        assert (out[-1] == 77).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,H,dropped,spare", LARGE)
def test_combine_backward_of_many_tokens_and_wide_rows(gpu_lib, T, k, H, dropped, spare):
    """A dot product goes over H / 2048 pieces of a row in at most H / 256 / 8 + 8 additions of a lane and the joins of
    ten steps and 16 waves: (H / 16 + 40) 2^-24 of the sum of magnitudes covers it."""
    g, at, rows, t_of, j_of, r_of, free = _large(T, k, H, dropped, spare, T + k + H + 2)
    src, dout, w = _normal(g, rows, H), _normal(g, T, H), _normal(g, T, k, dtype=torch.float32)
    d, dw = _guarded(rows, H), torch.full((T * k + 1,), 77.0, device="cuda")
    moe.moe_combine_rows_bwd(dout, at, src=src, topk_w=w, dsrc=d[:-1], dw=dw[:-1].view(T, k))
    got = dw[:-1].view(T, k)
    assert dw[-1] == 77 and (d[-1] == 77).all() and (d[:-1][free] == 77).all()
    want_dw, size = torch.zeros(T, k, dtype=torch.float64, device="cuda"), torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        i = (j_of == j).nonzero()[:, 0]
        grad = dout[t_of[i]].double() * w[t_of[i], j, None].double()
        assert ((d[r_of[i]].double() - grad).abs() <= grad.abs() * (HALF + 2.0 ** -24)).all()
        terms = src[r_of[i]].double() * dout[t_of[i]].double()
        want_dw[t_of[i], j], size[t_of[i], j] = terms.sum(1), terms.abs().sum(1)
    assert ((got.double() - want_dw).abs() <= (H / 16 + 40) * 2.0 ** -24 * size).all()
    # each output alone, in place, and as codes of the rounded gradient: the same bits
    d2, dw2 = _guarded(rows, H), torch.empty(T, k, device="cuda")
    moe.moe_combine_rows_bwd(dout, at, topk_w=w, dsrc=d2[:-1])
    moe.moe_combine_rows_bwd(dout, at, src=src, topk_w=w, dw=dw2)
    assert torch.equal(d2, d) and torch.equal(dw2, got)
    buf = src.clone()
    moe.moe_combine_rows_bwd(dout, at, src=buf, topk_w=w, dsrc=buf, dw=dw2)
    assert torch.equal(buf[r_of], d[r_of]) and torch.equal(buf[free], src[free]) and torch.equal(dw2, got)
    nb = (H + 127) // 128
    q, s = torch.zeros(rows, H, dtype=torch.uint8, device="cuda"), torch.zeros(nb, rows, device="cuda")
    moe.moe_block_quantize(d[:-1], q, s)
    codes, scales = _guarded(rows, H, dtype=torch.uint8), torch.full((nb, rows), 77.0, device="cuda")
    moe.moe_combine_rows_bwd(dout, at, src=src, topk_w=w, dsrc=d2[:-1], codes=codes[:-1], scales=scales, dw=dw2)
    assert torch.equal(codes[r_of], q[r_of]) and torch.equal(scales[:, r_of], s[:, r_of])
    assert torch.equal(d2, d) and torch.equal(dw2, got)
    assert (codes[:-1][free] == 77).all() and (codes[-1] == 77).all() and (scales[:, free] == 77).all()


@pytest.mark.gpu
def test_gradients_against_differences(gpu_lib):
    """d/dw and d/dsrc of sum(out * dout): out is linear in each, so a difference of any step is exact up to
    the roundings of two outputs; w in steps of 1 and dout in {-1, 0, 1} make all values exact."""
    g = torch.Generator().manual_seed(5)
    T, k, H = 7, 3, 48
    at, rows = _table(g, T, k, 0.2, 1)
    src = torch.randint(-3, 4, (rows, H), generator=g).bfloat16()
    w = torch.randint(-2, 3, (T, k), generator=g).float()
    dout = torch.randint(-1, 2, (T, H), generator=g).bfloat16()

    def loss(s, ww):
        out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        moe.moe_combine_rows(s.cuda(), at.cuda(), out, topk_w=ww.cuda())
        return (out.cpu().double() * dout.double()).sum()

    dsrc, dw = torch.zeros(rows, H, dtype=torch.bfloat16, device="cuda"), torch.empty(T, k, device="cuda")
    moe.moe_combine_rows_bwd(dout.cuda(), at.cuda(), src=src.cuda(), topk_w=w.cuda(), dsrc=dsrc, dw=dw)
    base = loss(src, w)
    for t in range(T):
        for j in range(k):
            w2 = w.clone()
            w2[t, j] += 1
            assert loss(src, w2) - base == dw[t, j].item()
    for r, c in ((0, 0), (rows - 1, H - 1), (rows // 2, 17)):
        s2 = src.clone()
        s2[r, c] += 1
        assert loss(s2, w) - base == dsrc[r, c].item()
    # dispatch: x's gradient is the sum over its rows
    x = torch.randint(-3, 4, (T, H), generator=g).bfloat16()
    drows = torch.randint(-2, 3, (rows, H), generator=g).bfloat16()

    def loss_x(xx):
        out = torch.zeros(rows, H, dtype=torch.bfloat16, device="cuda")
        moe.moe_dispatch_rows(xx.cuda(), at.cuda(), dst=out)
        return (out.cpu().double() * drows.double()).sum()

    dx = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    moe.moe_combine_rows(drows.cuda(), at.cuda(), dx)
    for t, c in ((0, 0), (T - 1, H - 1), (3, 20)):
        x2 = x.clone()
        x2[t, c] += 1
        assert loss_x(x2) - loss_x(x) == dx[t, c].item()


@pytest.mark.gpu
def test_spoilt_rows_reach_their_own_tokens_only(gpu_lib):
    T, k, H = 6, 2, 64
    g = torch.Generator().manual_seed(6)
    at, rows = _table(g, T, k)
    src, w = _rand(g, rows, H), _rand(g, T, k, dtype=torch.float32)
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    moe.moe_combine_rows(src.cuda(), at.cuda(), out, topk_w=w.cuda())
    src2 = src.clone()
    src2[at[2, 1], 5] = float("inf")
    src2.view(torch.int16)[at[4, 0].item()] = 0x7fff  # NaNs of all ones
    out2 = torch.empty_like(out)
    moe.moe_combine_rows(src2.cuda(), at.cuda(), out2, topk_w=w.cuda())
    assert torch.isinf(out2[2, 5]) and torch.isnan(out2[4]).all()
    same = torch.ones(T, H, dtype=torch.bool)
    same[2, 5] = False
    same[4] = False
    assert torch.equal(out.cpu()[same], out2.cpu()[same])


@pytest.mark.gpu
def test_after_the_dispatch_layout(gpu_lib):
    """The table as moe_dispatch_layout writes it, its error report included: then no row is named twice or
    outside, so nothing is written there."""
    T, H, E, k = 100, 64, 8, 3
    cfg = moe.make_cfg(T, H, 64, E, k)
    g = torch.Generator().manual_seed(8)
    idx = torch.argsort(torch.rand(T, E, generator=g), 1)[:, :k].int()
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, offsets, row_token, tok_row = (torch.empty(n, **i32) for n in (E, E + 1, T * k, (T, k)))
    moe.moe_dispatch_layout(cfg, idx.cuda(), counts, offsets, row_token, tok_row)
    x = _rand(g, T, H).cuda()
    rows = torch.empty(T * k, H, dtype=torch.bfloat16, device="cuda")
    moe.moe_dispatch_rows(x, tok_row, dst=rows)
    assert torch.equal(rows, x[row_token.long()])
    out = torch.empty_like(x)
    moe.moe_combine_rows(rows, tok_row, out)
    want = sum(x.float() for _ in range(k)).bfloat16()
    assert torch.equal(out, want)


@pytest.mark.gpu
def test_offsets_past_32_bits(gpu_lib):
    """Rows whose bytes lie past 2^32: the last ones of 2^32 / 2048 / 2 + 64 rows of 2048."""
    H = 2048
    R = (1 << 32) // (2 * H) + 64
    rows = torch.zeros(R, H, dtype=torch.bfloat16, device="cuda")
    T, k = 8, 4
    at = (R - T * k + torch.arange(T * k).view(T, k)).int().cuda()
    x = _rand(torch.Generator().manual_seed(9), T, H).cuda()
    moe.moe_dispatch_rows(x, at, dst=rows)
    assert torch.equal(rows[-T * k:], x.repeat_interleave(k, 0)) and not rows[:64].any()
    out = torch.empty_like(x)
    moe.moe_combine_rows(rows, at, out, topk_w=torch.full((T, k), 0.25, device="cuda"))
    assert torch.equal(out, x)
    dw = torch.empty(T, k, device="cuda")
    moe.moe_combine_rows_bwd(x, at, src=rows, dsrc=rows, dw=dw)  # (in place: every row of x is its own gradient)
    want = (x.double() ** 2).sum(1, keepdim=True).expand(T, k)
    assert ((dw.double() / want - 1).abs() < 1e-5).all() and torch.equal(rows[-T * k:], x.repeat_interleave(k, 0))


@pytest.mark.gpu
def test_captured_and_on_another_stream(gpu_lib):
    g = torch.Generator().manual_seed(10)
    T, k, H = 50, 4, 256
    at, rows = _table(g, T, k)
    at = at.cuda()
    x, w = _rand(g, T, H).cuda(), _rand(g, T, k, dtype=torch.float32).cuda()
    buf, out = torch.empty(rows, H, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    d, dw = torch.empty_like(buf), torch.empty_like(w)

    def step():
        moe.moe_dispatch_rows(x, at, dst=buf)
        moe.moe_combine_rows(buf, at, out, topk_w=w)
        moe.moe_combine_rows_bwd(out, at, src=buf, topk_w=w, dsrc=d, dw=dw)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (buf, out, d, dw)]
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((buf, out, d, dw), want))
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t in (buf, out, d, dw):
            t.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((buf, out, d, dw), want))
