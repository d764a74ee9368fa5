"""The layer for a few tokens (moe_layer_fwd_few): its refusals on the CPU, and on
the GPU its outputs against the layer in 64 bits within a derived bound."""
import ctypes

import numpy as np
import pytest
import torch

import dispatch_grouped_gemm_moe_amd as moe
from few_reference import few_layer
from moe_inputs import Workload, make_inputs

FAKE = 1 << 20  # aligned and never dereferenced: the checks fail first


def _cfg(T=8, H=128, I=64, E=8, k=2, **kw):
    return moe.make_cfg(T, H, I, E, k, **kw)


# ------------------------------------------------------------------ refusals (no GPU)

@pytest.mark.parametrize("kw,want", [
    (dict(T=0), moe.MOE_E_INVALID), (dict(k=9), moe.MOE_E_INVALID), (dict(H=96), moe.MOE_E_UNSUPPORTED),
    (dict(T=65), moe.MOE_E_UNSUPPORTED), (dict(flags=moe.MOE_F_IDENTITY_EXPERTS), moe.MOE_E_UNSUPPORTED)])
def test_few_refuses_configurations(kw, want):
    with pytest.raises(moe.MoeError) as e:
        moe.moe_query_few(_cfg(**kw))
    assert e.value.status == want


@pytest.mark.parametrize("kw", [dict(T=1, E=256, H=32704), dict(T=1, E=256, H=32768), dict(T=1, E=256, I=16384),
                                dict(T=1, E=128, H=32768, I=8128), dict(T=1, E=2, H=32768, I=32768),
                                dict(T=1, E=8, H=1 << 20, I=960), dict(T=64, E=8, H=1 << 20, I=1024), dict(minibatch=-1),
                                dict(T=1, E=240, H=32768, flags=moe.MOE_F_SHARED_EXPERT)])
@pytest.mark.parametrize("prec", [moe.MOE_PREC_BF16, moe.MOE_PREC_MXFP8])
def test_few_takes_the_configurations_that_the_weights_can_be_packed_for(kw, prec):
    cfg = _cfg(prec=prec, **kw)
    n = ctypes.c_size_t()
    assert moe.lib().moe_query_few(ctypes.byref(cfg), ctypes.byref(n)) == moe.moe_validate_cfg(cfg)


def test_few_workspace_depends_on_the_layer_only():
    base = moe.moe_query_few(_cfg())
    assert base % 256 == 0 and base >= 8 * 2 * 128 * 4
    assert moe.moe_query_few(_cfg(minibatch=4, ring_slots=2, comm_cus=8)) == base
    assert moe.moe_query_few(_cfg(T=64)) > base
    assert moe.moe_query_few(_cfg(flags=moe.MOE_F_SHARED_EXPERT)) > base
    assert moe.lib().moe_query_few(ctypes.byref(_cfg()), None) == moe.MOE_E_INVALID


def _call(cfg, ws_bytes=None, packed_bytes=None, **over):
    a = dict(x=FAKE, xc=None, xs=None, out=FAKE, ws=FAKE, Wr=FAKE, packed=FAKE, bias=None)
    a.update(over)
    s = moe.moe_query_sizes(_cfg(prec=cfg.prec, flags=cfg.flags))
    w = moe.moe_weights(a["Wr"], a["bias"], a["packed"], s.packed_weights if packed_bytes is None else packed_bytes)
    return moe.lib().moe_layer_fwd_few(ctypes.byref(cfg), ctypes.byref(w), a["x"], a["xc"], a["xs"], a["out"], a["ws"],
                                       1 << 40 if ws_bytes is None else ws_bytes, None)


@pytest.mark.parametrize("over", [dict(x=None), dict(out=None), dict(ws=None), dict(Wr=None), dict(packed=None),
                                  dict(x=FAKE + 8), dict(out=FAKE + 2), dict(ws=FAKE + 128), dict(packed=FAKE + 16),
                                  dict(Wr=FAKE + 2), dict(bias=FAKE + 1), dict(xc=FAKE), dict(xs=FAKE),
                                  dict(xc=FAKE, xs=FAKE)])
def test_few_refuses_pointers(over):
    assert _call(_cfg(), **over) == moe.MOE_E_INVALID


def test_few_refuses_small_buffers_and_misaligned_codes():
    cfg = _cfg(prec=moe.MOE_PREC_MXFP8)
    assert _call(cfg, xc=FAKE + 8, xs=FAKE) == moe.MOE_E_INVALID
    assert _call(cfg, xc=FAKE, xs=FAKE + 2) == moe.MOE_E_INVALID
    assert _call(cfg, ws_bytes=moe.moe_query_few(cfg) - 1) == moe.MOE_E_WORKSPACE
    s = moe.moe_query_sizes(cfg)
    assert _call(cfg, packed_bytes=s.packed_weights - 1) == moe.MOE_E_WORKSPACE


def test_few_binding_refuses_host_tensors():
    cfg = _cfg()
    u8, b16 = torch.uint8, torch.bfloat16
    with pytest.raises(moe.MoeError) as e:
        moe.moe_layer_fwd_few(cfg, torch.zeros(128, 8), None,
                              torch.zeros(moe.moe_query_sizes(cfg).packed_weights, dtype=u8),
                              torch.zeros(8, 128, dtype=b16), torch.zeros(8, 128, dtype=b16),
                              torch.zeros(moe.moe_query_few(cfg), dtype=u8), stream=0)
    assert e.value.status == moe.MOE_E_INVALID


def test_few_binding_refuses_tensors_the_kernels_cannot_read():
    cfg = _cfg()
    ok = dict(Wr=torch.zeros(128, 8), bias=None, packed=torch.zeros(16, dtype=torch.uint8),
              x=torch.zeros(8, 128, dtype=torch.bfloat16), out=torch.zeros(8, 128, dtype=torch.bfloat16),
              ws=torch.zeros(16, dtype=torch.uint8))
    bad = [dict(x=torch.zeros(8, 128)), dict(x=torch.zeros(128, 8, dtype=torch.bfloat16).t()),
           dict(out=torch.zeros(7, 128, dtype=torch.bfloat16)), dict(Wr=torch.zeros(127, 8)),
           dict(bias=torch.zeros(8, dtype=torch.float64)), dict(x_codes=torch.zeros(8, 64, dtype=torch.uint8)),
           dict(x=torch.zeros(8, 128, dtype=torch.bfloat16, device="meta"))]
    for b in bad:
        with pytest.raises(moe.MoeError) as e:
            moe.moe_layer_fwd_few(cfg, stream=0, **{**ok, **b})
        assert e.value.status == moe.MOE_E_INVALID, b


# ------------------------------------------------------------------ GPU

class Few:
    """One layer on the GPU, with a workspace whose contents past the counters are noise."""

    def __init__(self, w, inp=None):
        self.w, self.inp = w, inp or make_inputs(w)
        self.cfg = moe.make_cfg(w.T, w.H, w.I, w.E, w.k, prec=moe.MOE_PREC_MXFP8 if w.prec == "mxfp8" else 0,
                                flags=moe.MOE_F_SHARED_EXPERT if w.shared_expert else 0)
        d = lambda t: None if t is None else t.cuda().contiguous()
        i = self.inp
        self.Wr, self.bias, self.x = d(i.Wr), d(i.bias), d(i.x)
        self.packed = torch.empty(moe.moe_query_sizes(self.cfg).packed_weights, dtype=torch.uint8, device="cuda")
        moe.moe_prepare_weights(self.cfg, d(i.Wg), d(i.Wu), d(i.Wd), self.packed, d(i.Wsg), d(i.Wsu), d(i.Wsd))
        self.ws = torch.randint(0, 256, (moe.moe_query_few(self.cfg),), dtype=torch.uint8, device="cuda")
        self.ws[:moe.MOE_FEW_COUNTER_BYTES] = 0
        torch.cuda.synchronize()

    def __call__(self, x=None, **kw):
        x = self.x if x is None else x
        out = torch.full((x.shape[0] + 1, x.shape[1]), 7.0, dtype=torch.bfloat16, device="cuda")
        moe.moe_layer_fwd_few(self.cfg, self.Wr, self.bias, self.packed, x, out, self.ws, **kw)
        torch.cuda.synchronize()
        assert not self.ws[:moe.MOE_FEW_COUNTER_BYTES].any(), "the counters are not back at zero"
        assert (out[-1] == 7).all(), "a row past the last token was written"
        return out[:-1]


def _wl(T, H, I, E, k, prec="bf16", shared=False, bias="none", **kw):
    name = "few_%d_%d_%d_%d_%d_%s_%d" % (T, H, I, E, k, prec, shared)
    return Workload(name, T=T, H=H, I=I, E=E, k=k, prec=prec, shared_expert=shared, router_bias=bias,
                    stream=9000 + sum(map(ord, name)) % 997, **kw)


SHAPES = [(1, 64, 64, 1, 1), (1, 128, 64, 8, 2), (2, 2112, 128, 5, 3), (5, 192, 320, 6, 3), (7, 448, 64, 256, 16),
          (16, 320, 192, 4, 4), (17, 256, 128, 8, 2), (31, 128, 192, 7, 1), (33, 448, 320, 16, 5), (48, 64, 128, 2, 1),
          (64, 128, 64, 1, 1), (64, 4160, 64, 3, 2), (64, 192, 64, 200, 16), (9, 256, 1984, 8, 4), (16, 2240, 192, 6, 2),
          (7, 8256, 64, 1, 1), (4, 4160, 192, 6, 2), (50, 6208, 128, 2, 2), (1, 3136, 64, 32, 5)]


@pytest.mark.gpu
@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_few_matches_the_layer_in_64_bits(gpu_lib, shape, prec):
    w = _wl(*shape, prec=prec, shared=sum(shape) % 2 == 0, bias="normal" if shape[0] % 3 else "none")
    few = Few(w)
    got = few().double().cpu().numpy()
    ref, bound = few_layer(few.inp, w.T)
    worst = (np.abs(got - ref) / bound).max()
    print("%s: largest error %.3f of its bound" % (w.name, worst))
    assert worst <= 1


@pytest.mark.gpu
@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
def test_few_wide_magnitudes_and_skewed_routing(gpu_lib, prec):
    w = _wl(40, 256, 128, 12, 4, prec=prec, bias="zipf", wide_range=True)
    few = Few(w)
    ref, bound = few_layer(few.inp, w.T)
    assert (np.abs(few().double().cpu().numpy() - ref) <= bound).all()


@pytest.mark.gpu
def test_few_router_weight_off_16_bytes(gpu_lib):
    w = _wl(9, 192, 64, 8, 2)
    few = Few(w)
    want = few()
    shifted = torch.empty(few.Wr.numel() + 1, device="cuda")[1:].view(few.Wr.shape)
    shifted.copy_(few.Wr)
    few.Wr = shifted
    assert torch.equal(few(), want)


@pytest.mark.gpu
def test_few_ties_go_to_the_lower_expert(gpu_lib):
    w = _wl(6, 128, 64, 8, 2)
    inp = make_inputs(w)
    inp.Wr[:] = inp.Wr[:, :1]  # every logit of a token is the same: experts 0 and 1
    few = Few(w, inp)
    ref, bound = few_layer(inp, w.T)
    assert (np.abs(few().double().cpu().numpy() - ref) <= bound).all()
    inp.bias = torch.zeros(8)
    inp.bias[7] = 1.0
    few = Few(w, inp)
    ref, bound = few_layer(inp, w.T)
    assert (np.abs(few().double().cpu().numpy() - ref) <= bound).all()


@pytest.mark.gpu
@pytest.mark.parametrize("repeat", [1, 3, 50, 64, 70])
def test_few_ties_among_many_experts(gpu_lib, repeat):
    # expert e has the logit of expert e % repeat
    w = _wl(6, 128, 64, 200, 9)
    inp = make_inputs(w)
    inp.Wr = inp.Wr[:, torch.arange(200) % repeat].contiguous()
    few = Few(w, inp)
    ref, bound = few_layer(inp, w.T)
    assert (np.abs(few().double().cpu().numpy() - ref) <= bound).all()


@pytest.mark.gpu
@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
def test_few_reads_nothing_of_an_expert_that_no_token_chose(gpu_lib, prec):
    w = _wl(4, 128, 64, 6, 2, prec=prec)
    inp = make_inputs(w)
    inp.bias = torch.tensor([0.0, -1e4, 0.0, 0.0, -1e4, 0.0])
    clean = Few(w, inp)()
    for m in (inp.Wg, inp.Wu, inp.Wd):
        m[1], m[4] = 3e38, -3e38
    assert torch.equal(Few(w, inp)(), clean) and torch.isfinite(clean).all()


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_few_a_token_that_is_not_finite_spoils_only_itself(gpu_lib, bad):
    w = _wl(20, 256, 64, 8, 3)
    few = Few(w)
    want = few()
    x = few.x.clone()
    x[3, 17] = bad
    got = few(x)
    keep = torch.arange(20, device="cuda") != 3
    assert torch.equal(got[keep], want[keep]) and not torch.isfinite(got[3]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("T", [12, 20])
def test_few_mxfp8_token_that_is_not_finite_spoils_only_itself(gpu_lib, T, bad):
    # every expert is chosen by every token, so that the sums of the others keep their order
    w = _wl(T, 256, 64, 4, 4, prec="mxfp8", shared=True)
    few = Few(w)
    want = few()
    x = few.x.clone()
    x[3, 17] = bad
    got = few(x)
    keep = torch.arange(T, device="cuda") != 3
    assert torch.equal(got[keep], want[keep]) and not torch.isfinite(got[3]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("I", [64, 192, 448])
@pytest.mark.parametrize("T", [3, 20])
def test_few_an_infinite_weight_gives_infinity(gpu_lib, T, I):
    # the last row of Wd: steps past the end of I must not meet it again
    w = _wl(T, 128, I, 4, 4)
    inp = make_inputs(w)
    inp.x[:, 0] = 8  # gate and up of the last column are 8, so that h there is positive
    for m in (inp.Wg, inp.Wu):
        m[:, :, I - 1] = 0
        m[:, 0, I - 1] = 1
    clean = Few(w, inp)
    inp.Wd[:, I - 1, 5] = float("inf")
    few = Few(w, inp)
    got, want = few(), clean()
    other = torch.arange(128, device="cuda") != 5
    assert torch.equal(got[:, other], want[:, other])
    # h of the last column is positive for every token and expert: +inf, not NaN
    assert (got[:, 5] == float("inf")).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(3, 8, 2), (12, 2, 2), (16, 40, 2), (20, 4, 1), (40, 2, 2), (64, 48, 2)])
def test_few_an_infinite_weight_times_an_exact_h(gpu_lib, T, E, k):
    # h is 1 in its first column, which one bf16 value holds: neither of its parts may be zero
    w = _wl(T, 128, 64, E, k)
    inp = make_inputs(w)
    inp.x[:, 0] = 1
    for m in (inp.Wg, inp.Wu, inp.Wd):
        m.zero_()
    inp.Wg[:, 0, 0], inp.Wu[:, 0, 0] = 64, 1 / 64
    for e in range(E):
        inp.Wd[e, 0, e] = float("inf") if e % 2 else float("-inf")
    few = Few(w, inp)
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    moe.moe_route(few.cfg, few.x, few.Wr, few.bias, idx, torch.empty(T, k, device="cuda"))
    sign = torch.where(idx % 2 == 1, float("inf"), float("-inf")).bfloat16()
    want = torch.zeros(T, 128, dtype=torch.bfloat16, device="cuda").scatter_(1, idx.long(), sign)
    assert torch.equal(few(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
@pytest.mark.parametrize("shape", [(1, 448, 64, 256, 16), (6, 64, 64, 8, 3), (11, 2112, 64, 33, 7), (64, 320, 128, 256, 16)],
                         ids=lambda s: "-".join(map(str, s)))
def test_few_routes_as_the_router_does(gpu_lib, shape, prec):
    # silu(64) / 64 is 1 in fp32: expert e's output is 1 in column e, the layer's the routing weights
    w = _wl(*shape, prec=prec, bias="normal")
    inp = make_inputs(w)
    inp.x[:, 0] = 1
    for m in (inp.Wg, inp.Wu, inp.Wd):
        m.zero_()
    inp.Wg[:, 0, 0], inp.Wu[:, 0, 0] = 64, 1 / 64
    for e in range(w.E):
        inp.Wd[e, 0, e] = 1
    few = Few(w, inp)
    idx = torch.empty(w.T, w.k, dtype=torch.int32, device="cuda")
    gw = torch.empty(w.T, w.k, device="cuda")
    moe.moe_route(few.cfg, few.x, few.Wr, few.bias, idx, gw)
    want = torch.zeros(w.T, w.H, device="cuda").scatter_(1, idx.long(), gw).bfloat16()
    assert torch.equal(few(), want)


@pytest.mark.gpu
def test_few_codes_given_equal_codes_made(gpu_lib):
    for H in (320, 512):
        w = _wl(11, H, 128, 8, 2, prec="mxfp8", shared=True)
        few = Few(w)
        want = few()
        idx = torch.empty(w.T, w.k, dtype=torch.int32, device="cuda")
        gw = torch.empty(w.T, w.k, device="cuda")
        codes = torch.empty(w.T, H, dtype=torch.uint8, device="cuda")
        scales = torch.empty((H + 127) // 128, w.T, 4, dtype=torch.uint8, device="cuda")
        moe.moe_route(few.cfg, few.x, few.Wr, None, idx, gw, x_codes=codes, x_scales=scales)
        assert torch.equal(few(x_codes=codes, x_scales=scales), want)


@pytest.mark.gpu
@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
def test_few_agrees_with_the_layer_forward(gpu_lib, prec):
    # both are within the bound of the 64-bit layer; the layer forward also
    # rounds every expert's output to bf16 before the weighted sum
    w = _wl(33, 256, 192, 8, 4, prec=prec, shared=True)
    few = Few(w)
    ref, bound = few_layer(few.inp, w.T)
    ws = torch.zeros(moe.moe_query_sizes(few.cfg).workspace_fwd, dtype=torch.uint8, device="cuda")
    full = torch.empty_like(few.x)
    moe.moe_layer_fwd(few.cfg, few.Wr, few.bias, few.packed, few.x, full, ws)
    got = few().double().cpu().numpy()
    assert (np.abs(got - ref) <= bound).all()
    gap = np.abs(got - full.double().cpu().numpy()).max() / np.abs(ref).max()
    assert gap <= 2 * 2.0 ** -6, gap


@pytest.mark.gpu
def test_few_one_workspace_serves_calls_of_other_sizes(gpu_lib):
    a, b = Few(_wl(64, 256, 128, 16, 4, shared=True)), Few(_wl(3, 128, 64, 8, 2, prec="mxfp8"))
    want = a().clone(), b().clone()
    a.ws = b.ws = max(a.ws, b.ws, key=lambda t: t.numel())
    for _ in range(3):
        assert torch.equal(a(), want[0]) and torch.equal(b(), want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
def test_few_captured_twice_on_one_workspace(gpu_lib, prec):
    few = Few(_wl(10, 256, 128, 8, 2, prec=prec, shared=True))
    x1, x2 = few.x.clone(), few.x.flip(0).contiguous()
    want = [few(x1).clone(), few(x2).clone()]
    outs = [torch.empty_like(few.x) for _ in want]
    graphs = []
    for x, o in zip((x1, x2), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.moe_layer_fwd_few(few.cfg, few.Wr, few.bias, few.packed, x, o, few.ws)
        graphs.append(g)
    for i in (0, 1, 1, 0, 1):
        outs[i].zero_()
        graphs[i].replay()
        few(x2)  # the program's own call between replays
        assert torch.equal(outs[i], want[i])
    x1.copy_(x2)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[1])


@pytest.mark.gpu
def test_few_on_another_stream(gpu_lib):
    few = Few(_wl(12, 512, 256, 8, 2))
    want = few()
    s = torch.cuda.Stream()
    x = torch.zeros_like(few.x)
    torch.cuda.synchronize()
    out = torch.empty_like(x)
    with torch.cuda.stream(s):
        torch.cuda._sleep(1000000)
        x.copy_(few.x)
        moe.moe_layer_fwd_few(few.cfg, few.Wr, few.bias, few.packed, x, out, few.ws)
    s.synchronize()
    assert torch.equal(out, want)


@pytest.mark.gpu
def test_few_two_calls_at_once(gpu_lib):
    few = [Few(_wl(12, 512, 256, 8, 2, prec="mxfp8")), Few(_wl(40, 512, 256, 8, 3))]
    want = [f() for f in few]
    outs = [torch.zeros_like(f.x) for f in few]
    streams = [torch.cuda.Stream() for _ in few]
    torch.cuda.synchronize()
    for _ in range(20):
        for f, o, s in zip(few, outs, streams):
            moe.moe_layer_fwd_few(f.cfg, f.Wr, f.bias, f.packed, f.x, o, f.ws, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("T,prec", [(1, "bf16"), (20, "bf16"), (2, "mxfp8")])
def test_few_weights_past_32_bits(gpu_lib, T, prec):
    # the bias sends every token to the last two experts; alone they are the same layer
    H, I, E = 8192, 2112, 66 if prec == "bf16" else 132  # gate and up of every expert: 2^32 bytes and more
    g = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)
    Wg, Wu, Wd = (torch.zeros(E, *s, device="cuda", dtype=torch.bfloat16) for s in ((H, I), (H, I), (I, H)))
    for m in (Wg, Wu, Wd):
        m[-2:] = rand(2, *m.shape[1:]) / 64
    x, Wr = rand(T, H), torch.randn(H, E, generator=g, device="cuda") / 64
    bias = torch.full((E,), -1e4, device="cuda")
    bias[-2:] = 0
    got = []
    for n in (E, 2):
        cfg = moe.make_cfg(T, H, I, n, 2, prec=moe.MOE_PREC_MXFP8 if prec == "mxfp8" else 0)
        packed = torch.empty(moe.moe_query_sizes(cfg).packed_weights, dtype=torch.uint8, device="cuda")
        moe.moe_prepare_weights(cfg, *(m[-n:].contiguous() for m in (Wg, Wu, Wd)), packed)
        ws = torch.zeros(moe.moe_query_few(cfg), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(x)
        moe.moe_layer_fwd_few(cfg, Wr[:, -n:].contiguous(), bias[-n:].contiguous(), packed, x, out, ws)
        torch.cuda.synchronize()
        got.append(out)
        del packed
    assert got[0].abs().max() > 0.01 and torch.isfinite(got[0]).all()
    assert torch.equal(got[0], got[1])


@pytest.mark.gpu
def test_few_buffers_of_any_type(gpu_lib):
    # moe_prepare_weights and moe_layer_fwd take packed weights and a workspace of any type, by their bytes
    few = Few(_wl(5, 128, 64, 8, 2, prec="mxfp8"))
    want = few()

    def call(packed, ws):
        out = torch.zeros_like(few.x)
        moe.moe_layer_fwd_few(few.cfg, few.Wr, few.bias, packed, few.x, out, ws)
        torch.cuda.synchronize()
        return out

    for dtype in (torch.int8, torch.bfloat16, torch.int64):
        packed, ws = few.packed.view(dtype), few.ws.view(dtype)
        assert torch.equal(call(packed, ws), want)
        for short in ((packed[:-1], ws), (packed, ws[:-1])):
            with pytest.raises(moe.MoeError) as e:
                call(*short)
            assert e.value.status == moe.MOE_E_WORKSPACE


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 20])
@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
def test_few_a_nan_of_any_payload_spoils_its_token(gpu_lib, prec, T):
    w = _wl(T, 256, 64, 4, 4, prec=prec, shared=True)  # every expert: the others' sums keep their order
    few = Few(w)
    want = few()
    keep = torch.arange(T, device="cuda") != 3
    for bits in (0x7FFF, -1, 0x7F81, -0x7F, 0x7FC0):
        x = few.x.clone()
        x.view(torch.int16)[3, 17] = bits
        got = few(x)
        assert torch.isnan(got[3]).all() and torch.equal(got[keep], want[keep]), hex(bits)
