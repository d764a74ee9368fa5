"""The global gradient norm and clipping (moe_grad_norm, moe_clip_grads): refusals on the CPU, and on the
GPU the norm against a 64-bit sum and the clipped gradients against it.

Bounds.  The norm is a 64-bit sum rounded to fp32 once: 2^-24 of it (and 2^-40 for the sum's own roundings).
The factor is rounded once more and so is every product: 3 * 2^-24 in fp32, and 2^-8 in bf16."""
import ctypes

import pytest
import torch

import dispatch_grouped_gemm_moe_amd as moe

FAKE = 1 << 20


def _arrays(ptrs, counts, kinds=None):
    n = len(ptrs)
    return ((ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*counts),
            None if kinds is None else (ctypes.c_uint8 * n)(*kinds))


def _norm(ptrs=(FAKE, FAKE), counts=(5, 6), kinds=None, tensors=None, norm=FAKE, ws=FAKE, ws_bytes=1 << 30):
    p, c, k = _arrays(ptrs, counts, kinds)
    return moe.lib().moe_grad_norm(len(ptrs) if tensors is None else tensors, p, c, k, norm, ws, ws_bytes, None)


def _clip(ptrs=(FAKE, FAKE), counts=(5, 6), kinds=None, tensors=None, norm=FAKE, max_norm=1.0, out=(FAKE, FAKE)):
    p, c, k = _arrays(ptrs, counts, kinds)
    o = None if out is None else (ctypes.c_void_p * len(out))(*out)
    return moe.lib().moe_clip_grads(len(ptrs) if tensors is None else tensors, p, c, k, norm, max_norm, o, None)


BAD = [dict(tensors=0), dict(tensors=-1), dict(ptrs=(FAKE, None)), dict(ptrs=(FAKE, FAKE + 2)),
       dict(ptrs=(FAKE + 1, FAKE), kinds=(1, 0)), dict(counts=(5, -1)), dict(norm=None), dict(norm=FAKE + 2)]


@pytest.mark.parametrize("kw", BAD + [dict(ws=None), dict(ws=FAKE + 8)])
def test_norm_refuses(kw):
    assert _norm(**kw) == moe.MOE_E_INVALID


@pytest.mark.parametrize("kw", BAD + [dict(out=None), dict(out=(FAKE, None)), dict(out=(FAKE, FAKE + 2)),
                                      dict(max_norm=0.0), dict(max_norm=-1.0), dict(max_norm=float("nan"))])
def test_clip_refuses(kw):
    assert _clip(**kw) == moe.MOE_E_INVALID


def test_limits_and_workspace():
    assert _norm(counts=(5, (1 << 48) + 1)) == _clip(counts=(5, (1 << 48) + 1)) == moe.MOE_E_UNSUPPORTED
    assert _norm(ws_bytes=moe.moe_query_grad_norm(2) - 1) == moe.MOE_E_WORKSPACE
    assert moe.lib().moe_query_grad_norm(1, None) == moe.MOE_E_INVALID
    for n, want in ((0, moe.MOE_E_INVALID), (-1, moe.MOE_E_INVALID), ((1 << 20) + 1, moe.MOE_E_UNSUPPORTED),
                    (1 << 32, moe.MOE_E_INVALID)):
        with pytest.raises(moe.MoeError) as e:
            moe.moe_query_grad_norm(n)
        assert e.value.status == want
    null = ctypes.c_void_p()
    assert moe.lib().moe_grad_norm(1, null, null, null, FAKE, FAKE, 1 << 30, None) == moe.MOE_E_INVALID


def test_binding_refuses_tensors_the_kernels_cannot_read():
    f, b = torch.zeros(8), torch.zeros(8, dtype=torch.bfloat16)
    norm, ws = torch.zeros(1), torch.zeros(1 << 16, dtype=torch.uint8)
    for grads in ([f], [], [f.double()], [torch.zeros(8, 2)[:, 0]], [f.to("meta")], [f.half()]):
        with pytest.raises(moe.MoeError) as e:  # (the first: host tensors)
            moe.moe_grad_norm(grads, norm, ws, stream=0)
        assert e.value.status == moe.MOE_E_INVALID
    for out in ([f], [f, f], [f, b[:4]], [b, f]):
        with pytest.raises(moe.MoeError) as e:
            moe.moe_clip_grads([f, b], norm, 1.0, out=out, stream=0)
        assert e.value.status == moe.MOE_E_INVALID


# ------------------------------------------------------------------ GPU

def _ws(n):
    ws = torch.full((moe.moe_query_grad_norm(n),), 0xff, dtype=torch.uint8, device="cuda")
    ws[:moe.MOE_GRAD_COUNTER_BYTES] = 0
    return ws


def _grads(g, shapes, sigma=1.0):
    """Tensors of (elements, type, offset): `offset` elements into a buffer of their own."""
    out = []
    for n, dtype, off in shapes:
        buf = (torch.randn(n + off, generator=g) * sigma).to(dtype).cuda()
        out.append(buf[off:])
    return out


F, B = torch.float32, torch.bfloat16
CASES = [[(1, F, 0)], [(1, B, 0)], [(0, F, 0)], [(0, F, 0), (5, B, 1), (0, B, 0)], [(1023, F, 0), (1025, B, 0), (4096, F, 1)],
         [(100003, F, 0), (70001, B, 3), (1, F, 3)], [(i * 37 % 1500, B if i % 3 == 0 else F, i % 5) for i in range(250)],
         [(3_000_001, F, 0), (2_500_000, B, 0)], [(17, F, 0)] * 96, [(17, B, 0)] * 97]


def _want(grads):
    return sum((t.cpu().double() ** 2).sum() for t in grads).sqrt()


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(CASES)))
def test_norm_and_clip(gpu_lib, case):
    g = torch.Generator().manual_seed(case)
    grads = _grads(g, CASES[case])
    ws = _ws(len(grads))
    norm = torch.full((2,), 77.0, device="cuda")
    want = _want(grads)
    runs = []
    for _ in range(3):
        moe.moe_grad_norm(grads, norm, ws)
        torch.cuda.synchronize()
        runs.append(norm.cpu().clone())
        assert not ws[:moe.MOE_GRAD_COUNTER_BYTES].any()
    assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2]) and runs[0][1] == 77
    assert abs(runs[0][0].double() - want) <= want * (2.0 ** -24 + 2.0 ** -40)
    for max_norm in (float(want) * 0.3 + 1e-3, float(want) * 3 + 1, float("inf")):
        coef = min(1.0, max_norm / (float(norm[0]) + 1e-6))
        outs = [torch.full((t.numel() + 1,), 77, dtype=t.dtype, device="cuda") for t in grads]
        moe.moe_clip_grads(grads, norm, max_norm, out=[o[:-1] for o in outs])
        for t, o in zip(grads, outs):
            w, eps = t.cpu().double() * coef, 2.0 ** -8 if t.dtype is B else 2.0 ** -23
            tiny = 2.0 ** -133 if t.dtype is B else 2.0 ** -149
            assert ((o[:-1].cpu().double() - w).abs() <= w.abs() * (eps + 2.0 ** -24) + tiny).all()
            assert o[-1] == 77
            if coef == 1.0:
                assert torch.equal(o[:-1], t)
        inplace = [t.clone() for t in grads]
        moe.moe_clip_grads(inplace, norm, max_norm)
        assert all(torch.equal(a, o[:-1]) for a, o in zip(inplace, outs))


@pytest.mark.gpu
def test_squares_that_overflow_fp32(gpu_lib):
    grads = [torch.full((1000,), 3e38, device="cuda"), torch.full((1000,), 1e-30, device="cuda")]
    norm, ws = torch.empty(1, device="cuda"), _ws(2)
    moe.moe_grad_norm(grads, norm, ws)
    assert torch.isinf(norm).all()  # 9.5e39: past fp32, as a value; its square was not in the way
    moe.moe_grad_norm(grads[:1][0:1] and [torch.full((16,), 5e37, device="cuda")], norm, ws)
    assert abs(norm.item() / 2e38 - 1) < 1e-6
    moe.moe_grad_norm([torch.full((1 << 20,), 1e-30, device="cuda")], norm, ws)
    assert abs(norm.item() / 1.024e-27 - 1) < 1e-6


@pytest.mark.gpu
def test_nan_and_infinity(gpu_lib):
    norm, ws = torch.empty(1, device="cuda"), _ws(2)
    a, b = torch.ones(300, device="cuda"), torch.ones(200, dtype=B, device="cuda")
    b[7] = float("nan")
    moe.moe_grad_norm([a, b], norm, ws)
    assert torch.isnan(norm).all()
    moe.moe_clip_grads([a, b], norm, 1.0)
    assert torch.isnan(a).all() and torch.isnan(b).all()
    a, b = torch.ones(300, device="cuda"), torch.ones(200, dtype=B, device="cuda")
    a[299] = -float("inf")
    moe.moe_grad_norm([a, b], norm, ws)
    assert torch.isinf(norm).all() and norm.item() > 0
    moe.moe_clip_grads([a, b], norm, 1.0)
    assert torch.isnan(a[299]) and not a[:299].any() and not b.any()


@pytest.mark.gpu
def test_a_tensor_past_32_bits(gpu_lib):
    n = (1 << 32) // 2 + 1000  # bf16: past 2^32 bytes
    t = torch.zeros(n, dtype=B, device="cuda")
    t[0], t[-1] = 3, 4
    norm, ws = torch.empty(1, device="cuda"), _ws(1)
    moe.moe_grad_norm([t], norm, ws)
    assert norm.item() == 5
    moe.moe_clip_grads([t], norm, 2.5)
    assert t[0] == 1.5 and t[-1] == 2 and t.count_nonzero() == 2


@pytest.mark.gpu
def test_captured_replayed_and_on_another_stream(gpu_lib):
    g = torch.Generator().manual_seed(3)
    grads = _grads(g, [(5000, F, 0)] * 100 + [(70000, B, 0)])
    out = [torch.empty_like(t) for t in grads]
    norm, ws = torch.empty(1, device="cuda"), _ws(len(grads))

    def step():
        moe.moe_grad_norm(grads, norm, ws)
        moe.moe_clip_grads(grads, norm, 1.0, out=out)

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (norm, *out)]
    s = torch.cuda.Stream()
    norm.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((norm, *out), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        for t in grads:
            t.mul_(2 if i else 1)
        graph.replay()
        torch.cuda.synchronize()
        assert abs(norm.item() / (want[0].item() * 2 ** i) - 1) < 1e-6
        moe.moe_grad_norm(out, norm, ws)  # eager work on the same workspace, between replays
        assert abs(norm.item() - 1) < 2e-3
        assert not ws[:moe.MOE_GRAD_COUNTER_BYTES].any()


@pytest.mark.gpu
def test_two_calls_at_once(gpu_lib):
    """Norm and clipping of two lists on two streams, a workspace each, while the other's run: as alone."""
    g = torch.Generator().manual_seed(7)
    jobs = []
    for shapes in ([(3_000_001, F, 0), (70_000, B, 1)], [(5000, F, 0)] * 120):
        grads = _grads(g, shapes)
        out = [torch.empty_like(t) for t in grads]
        norm, ws = torch.empty(1, device="cuda"), _ws(len(grads))

        def run(stream, grads=grads, out=out, norm=norm, ws=ws):
            moe.moe_grad_norm(grads, norm, ws, stream=stream)
            moe.moe_clip_grads(grads, norm, 1.0, out=out, stream=stream)

        run(torch.cuda.current_stream())
        torch.cuda.synchronize()
        jobs.append((run, (norm, *out), [t.clone() for t in (norm, *out)], torch.cuda.Stream(), ws))
    for _, outs, *_ in jobs:
        for t in outs:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(30):
        for run, _, _, stream, _ in jobs:
            run(stream)
    torch.cuda.synchronize()
    for _, outs, alone, _, ws in jobs:
        assert all(torch.equal(x, y) for x, y in zip(outs, alone))
        assert not ws[:moe.MOE_GRAD_COUNTER_BYTES].any()


@pytest.mark.gpu
def test_after_the_layers_backward(gpu_lib):
    """The gradients of moe_layer_bwd, clipped together in place, as a training step does."""
    T, H, I, E, k = 64, 128, 64, 8, 2
    g = torch.Generator().manual_seed(4)
    cfg = moe.make_cfg(T, H, I, E, k)
    bufs = moe.alloc_buffers(cfg, with_saved=True)
    Wr = (torch.randn(H, E, generator=g) * 0.1).cuda()
    W = [(torch.randn(E, *s, generator=g) * 0.1).bfloat16().cuda() for s in ((H, I), (H, I), (I, H))]
    moe.moe_prepare_weights(cfg, *W, bufs.packed)
    x, dout = (torch.randn(T, H, generator=g).bfloat16().cuda() for _ in range(2))
    out, dx = torch.empty_like(x), torch.empty_like(x)
    grads = [torch.empty(w.shape, device="cuda") for w in W] + [torch.empty(H, E, device="cuda")]
    moe.moe_layer_fwd(cfg, Wr, None, bufs.packed, x, out, bufs.ws, saved=bufs.saved)
    moe.moe_layer_bwd(cfg, Wr, None, bufs.packed, x, dout, bufs.saved, dx, *grads, bufs.ws)
    norm, ws = torch.empty(1, device="cuda"), _ws(len(grads))
    want, before = _want(grads), [t.clone() for t in grads]
    moe.moe_grad_norm(grads, norm, ws)
    moe.moe_clip_grads(grads, norm, 0.5)
    assert abs(norm.item() - want) <= want * 2.0 ** -23
    for t, b in zip(grads, before):
        w = b.double() * (0.5 / (want.item() + 1e-6))
        assert ((t.double() - w).abs() <= w.abs() * 2.0 ** -22 + 2.0 ** -149).all()
    assert abs(_want(grads) - 0.5) < 1e-5
