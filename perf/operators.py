"""Cases of the operators around and inside the MoE layer of a transformer block.

    few       the whole layer for 1 to 64 tokens (moe_layer_fwd_few): router, SwiGLU
              experts and weighted sum, as a server runs it for every decoded token
    norm      the block's residual addition and root-mean-square norm in front of the
              layer (moe_add_rmsnorm_fwd), with the MXFP8 codes that the layer takes and
              the 8-bit checkpoint of the residual stream that a training run keeps;
              codes are read back by moe_mx_dequantize
    norm_bwd  its backward pass (moe_add_rmsnorm_bwd), from the bf16 residual stream or
              from the 8-bit checkpoint
    block     norm and few in a row: the MoE half of a block for a decode step

Values held in MXFP8 (E4M3 codes, one power-of-two scale per 32 elements) are returned
as the bf16 values that they stand for, which is exact.
"""
import math

import torch

own = False

EPS = 1e-5
LARGEST_WEIGHTS = 32 * 7168 * 2048  # elements of one of the largest listed layer's three weight stacks
LARGEST_ROWS = 16384 * 7168  # elements of the largest listed norm


def _few(name, T, H, I, E, k, prec="bf16", shared=False, bias=False):
    c = {"op": "few", "T": T, "H": H, "I": I, "E": E, "k": k, "prec": prec, "shared": shared, "bias": bias}
    return dict(c, name=name) if name else c


def _norm(name, op, rows, cols, residual=True, codes=False, checkpoint=False):
    c = {"op": op, "rows": rows, "cols": cols, "residual": residual, "codes": codes, "checkpoint": checkpoint}
    return dict(c, name=name) if name else c


def listed():
    return [
        # the smallest layer of this repository's tests: nothing but latency
        _few("few_t1_h128", 1, 128, 64, 8, 2),
        # one sequence being decoded, on a small and on the large layer shape
        _few("few_t1_h2048_e64", 1, 2048, 1024, 64, 6),
        _few("few_t1_h7168_mx", 1, 7168, 2048, 32, 8, prec="mxfp8", bias=True),
        # many small experts, an odd number of tokens
        _few("few_t7_e256_k16_mx", 7, 1024, 512, 256, 16, prec="mxfp8"),
        # a small serving batch with the shared expert
        _few("few_t16_h7168_mx_shared", 16, 7168, 2048, 32, 8, prec="mxfp8", shared=True),
        # the largest batch: every expert's weights are read
        _few("few_t64_h7168", 64, 7168, 2048, 32, 8, bias=True),
        # the norm of one decoded token, with the codes the MXFP8 layer takes
        _norm("norm_r1_h7168_mx", "norm", 1, 7168, codes=True),
        # a first block's norm (no residual) on ragged sizes
        _norm("norm_r999_h2080", "norm", 999, 2080, residual=False),
        # a training step's norm: codes for the layer, checkpoint for the backward pass
        _norm("norm_r16384_h7168_mx_ck", "norm", 16384, 7168, codes=True, checkpoint=True),
        # a training step's backward pass, from the bf16 stream and from the checkpoint
        _norm("bwd_r16384_h7168", "norm_bwd", 16384, 7168),
        _norm("bwd_r4096_h2048_ck", "norm_bwd", 4096, 2048, checkpoint=True),
        # the MoE half of a block for eight sequences being decoded
        dict(_few(None, 8, 2048, 1024, 64, 6, prec="mxfp8"), op="block", name="block_t8_h2048_mx"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["few", "few", "norm", "norm_bwd", "block"])
    if op in ("few", "block"):
        T, H, I, E = _log(rng, 1, 64), 64 * _log(rng, 2, 112), 64 * _log(rng, 1, 32), _log(rng, 1, 256)
        shared = rng.random() < 0.3
        while (E + shared) * H * I > LARGEST_WEIGHTS:
            E = E // 2
        k = rng.randint(1, min(E, 16))
        prec = "mxfp8" if op == "block" else rng.choice(["bf16", "mxfp8"])
        return dict(_few(None, T, H, I, E, k, prec, shared, rng.random() < 0.5), op=op)
    rows, cols = _log(rng, 1, 16384), 32 * _log(rng, 2, 256)
    rows = min(rows, LARGEST_ROWS // cols)
    if op == "norm":
        return _norm(None, op, rows, cols, rng.random() < 0.7, rng.random() < 0.5, rng.random() < 0.3)
    return _norm(None, op, rows, cols, rng.random() < 0.7, False, rng.random() < 0.5)


def work(case):
    if case["op"] in ("few", "block"):
        T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
        # the experts that T tokens of k distinct choices each reach, as expected
        # of an even router; MXFP8 weights are a code and 1/32 of a scale each
        active = E * (1 - (1 - k / E) ** T)
        bits = 33 / 32 if case["prec"] == "mxfp8" else 2
        weights = 3 * H * I * (active * bits + 2 * case["shared"])
        data = T * H * (4 if case["op"] == "few" else 8)
        return {"bytes": weights + 4 * H * E + data, "flops": 6 * T * (k + case["shared"]) * H * I + 2 * T * H * E}
    n = case["rows"] * case["cols"]
    mx = 33 / 32
    if case["op"] == "norm":
        each = 2 + 2 + 4 * case["residual"] + mx * (case["codes"] + case["checkpoint"])
        return {"bytes": n * each, "flops": 6 * n}
    each = 2 + 2 + 2 * case["residual"] + (mx if case["checkpoint"] else 2)
    return {"bytes": n * each, "flops": 12 * n}


# ---------------------------------------------------------------- inputs


def _codes(v):
    """E4M3 codes and scale bytes of v (its last axis in blocks of 32): the scale 2^e is
    the smallest with max|block| <= 448 * 2^e, e = 0 for a block of zeros."""
    b = v.float().reshape(*v.shape[:-1], -1, 32)
    m, p = torch.frexp(b.abs().amax(-1))
    e = torch.where(m > 0, p - 9 + (m > 0.875).int(), 0).clamp(-127, 127)
    q = torch.ldexp(b, -e[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).reshape(v.shape), (e + 127).to(torch.uint8)


def _values(codes, scales):
    """The bf16 values that codes and their scale bytes (one per 32) stand for."""
    b = codes.view(torch.float8_e4m3fn).float().reshape(*scales.shape, 32)
    return torch.ldexp(b, scales.int()[..., None] - 127).reshape(codes.shape).bfloat16()


def _held(w):
    """A weight stack [E, K, N] as MXFP8 along K holds it, by expert."""
    out = torch.empty_like(w)
    for e in range(w.shape[0]):
        out[e] = _values(*_codes(w[e].t().contiguous())).t()
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, sigma=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=dtype) * sigma)

    st = dict(case)
    if case["op"] in ("few", "block"):
        T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
        mx, shared = case["prec"] == "mxfp8", case["shared"]
        st["x"] = normal(T, H)
        if case["op"] == "block":
            st["residual"] = normal(T, H, sigma=4.0)
            st["gain"] = 1 + normal(H, sigma=0.1, dtype=torch.float32)
        st["Wr"] = normal(H, E, sigma=0.02, dtype=torch.float32)
        st["b"] = normal(E, dtype=torch.float32) if case["bias"] else None
        Wg, Wu, Wd = normal(E, H, I, sigma=0.02), normal(E, H, I, sigma=0.02), normal(E, I, H, sigma=0.02)
        Sg, Su, Sd = ((normal(H, I, sigma=0.02), normal(H, I, sigma=0.02), normal(I, H, sigma=0.02))
                      if shared else (None, None, None))
        if own:  # a server's program keeps the packed weights, laid out once, and a workspace
            import dispatch_grouped_gemm_moe_amd as moe
            cfg = moe.make_cfg(T, H, I, E, k, prec=moe.MOE_PREC_MXFP8 if mx else moe.MOE_PREC_BF16,
                               flags=moe.MOE_F_SHARED_EXPERT if shared else 0)
            st["cfg"] = cfg
            st["packed"] = torch.empty(moe.moe_query_sizes(cfg).packed_weights, dtype=torch.uint8, device="cuda")
            st["ws"] = torch.zeros(moe.moe_query_few(cfg), dtype=torch.uint8, device="cuda")
            moe.moe_prepare_weights(cfg, Wg, Wu, Wd, st["packed"], Sg, Su, Sd)
            torch.cuda.synchronize()
        else:  # the routed experts' weights as the layer's precision holds them
            st["W"] = [_held(w) for w in (Wg, Wu, Wd)] if mx else [Wg, Wu, Wd]
            st["S"] = [Sg, Su, Sd]
        return st
    rows, cols = case["rows"], case["cols"]
    st["gain"] = 1 + normal(cols, sigma=0.1, dtype=torch.float32)
    if case["op"] == "norm":
        st["x"] = normal(rows, cols)
        # the stream that many blocks have added to: larger than what one block adds
        st["residual"] = normal(rows, cols, sigma=4.0) if case["residual"] else None
        return st
    st["dy"] = normal(rows, cols)
    st["dsum"] = normal(rows, cols) if case["residual"] else None
    s = normal(rows, cols, sigma=4.0)
    st["rstd"] = (s.double().square().mean(1) + EPS).rsqrt().float()
    if case["checkpoint"]:
        st["codes"], st["scales"] = _codes(s)
    else:
        st["s"] = s
    if own:
        import dispatch_grouped_gemm_moe_amd as moe
        st["ws"] = torch.empty(moe.moe_query_add_rmsnorm_bwd(rows, cols), dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------- the plain form


def _rounded(v):
    """v as MXFP8 along its last axis holds it (elementary operations, in v's type)."""
    b = v.reshape(*v.shape[:-1], -1, 32)
    m, p = torch.frexp(b.abs().amax(-1, keepdim=True))
    e = torch.where(m > 0, p - 9 + (m > 0.875).int(), 0).clamp(-127, 127)
    q = torch.ldexp(b, -e)
    # E4M3: three fraction bits, exponents from -6; 448 is the largest value
    step = torch.ldexp(torch.ones_like(q), torch.frexp(q)[1].clamp(min=-5) - 4)
    q = (torch.round(q / step) * step).clamp(-448, 448)
    return torch.ldexp(q, e).reshape(v.shape)


def _swiglu(g, u):
    return g / (1 + torch.exp(-g)) * u


def _layer(st, x):
    T, E, k, mx = st["T"], st["E"], st["k"], st["prec"] == "mxfp8"
    hold = _rounded if mx else (lambda v: v)
    # the choice of experts is decided in 64 bits, ties to the lower index
    logits = x.double() @ st["Wr"].double()
    if st["b"] is not None:
        logits = logits + st["b"].double()
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    w = torch.exp(top - top[:, :1])
    w = (w / w.sum(1, keepdim=True)).float()
    xf = x.float()
    xq = hold(xf)
    Wg, Wu, Wd = st["W"]
    if T * k <= E:  # the chosen experts' weights, one copy per (token, choice)
        at = idx.reshape(-1)
        rows = xq.repeat_interleave(k, 0)[:, None, :]
        h = hold(_swiglu(rows @ Wg[at].float(), rows @ Wu[at].float()))
        y = (h @ Wd[at].float()).reshape(T, k, -1)
    else:  # every expert for every token
        h = hold(_swiglu(xq @ Wg.float(), xq @ Wu.float()))
        y = (h @ Wd.float()).transpose(0, 1)
        y = y.gather(1, idx[:, :, None].expand(T, k, y.shape[2]))
    out = (w[:, :, None] * y).sum(1)
    if st["shared"]:  # always bf16 weights, unquantised
        Sg, Su, Sd = (s.float() for s in st["S"])
        out = out + _swiglu(xf @ Sg, xf @ Su) @ Sd
    return out.bfloat16()


def _normed(st):
    x, r = st["x"], st["residual"]
    s = x if r is None else (x.float() + r.float()).bfloat16()
    sf = s.float()
    rstd = 1 / torch.sqrt((sf * sf).mean(1) + EPS)
    y = (sf * rstd[:, None] * st["gain"]).bfloat16()
    return s, y, rstd


def _plain(st):
    if st["op"] == "few":
        return _layer(st, st["x"])
    if st["op"] == "block":
        s, y, _ = _normed(st)
        return {"sum": s, "out": _layer(st, y)}
    if st["op"] == "norm":
        s, y, rstd = _normed(st)
        out = {"y": y, "rstd": rstd}
        if st["residual"] is not None:
            out["sum"] = s
        if st["codes"]:
            out["y_held"] = _rounded(y.float()).bfloat16()
        if st["checkpoint"]:
            out["sum_held"] = _rounded(s.float()).bfloat16()
        return out
    s = _values(st["codes"], st["scales"]) if st["checkpoint"] else st["s"]
    dy, rstd = st["dy"].float(), st["rstd"][:, None]
    xhat = s.float() * rstd
    gy = dy * st["gain"]
    dx = rstd * (gy - xhat * (gy * xhat).mean(1, keepdim=True))
    if st["dsum"] is not None:
        dx = dx + st["dsum"].float()
    return {"dx": dx.bfloat16(), "dgain": (dy * xhat).sum(0)}


# ---------------------------------------------------------------- the framework's calls


def _own(st):
    import dispatch_grouped_gemm_moe_amd as moe
    if st["op"] == "few":
        out = torch.empty_like(st["x"])
        moe.moe_layer_fwd_few(st["cfg"], st["Wr"], st["b"], st["packed"], st["x"], out, st["ws"])
        return out
    if st["op"] == "norm_bwd":
        dx, dgain = torch.empty_like(st["dy"]), torch.empty_like(st["gain"])
        ck = st["checkpoint"]
        moe.moe_add_rmsnorm_bwd(st["dy"], st["gain"], st["rstd"], dx, dgain, st["ws"], summed=None if ck else st["s"],
                                ck_codes=st["codes"] if ck else None, ck_scales=st["scales"] if ck else None,
                                dsum=st["dsum"])
        return {"dx": dx, "dgain": dgain}
    x, r = st["x"], st["residual"]
    rows, cols = x.shape
    s, y = None if r is None else torch.empty_like(x), torch.empty_like(x)
    if st["op"] == "block":
        codes = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
        scales = torch.empty((cols + 127) // 128, rows, 4, dtype=torch.uint8, device="cuda")
        moe.moe_add_rmsnorm_fwd(x, st["gain"], y, eps=EPS, residual=r, summed=s, y_codes=codes, y_scales=scales)
        out = torch.empty_like(x)
        moe.moe_layer_fwd_few(st["cfg"], st["Wr"], st["b"], st["packed"], y, out, st["ws"], x_codes=codes,
                              x_scales=scales)
        return {"sum": s, "out": out}
    out = {"y": y, "rstd": torch.empty(rows, dtype=torch.float32, device="cuda")}
    more = {}
    if s is not None:
        out["sum"] = s
    if st["codes"]:
        more["y_codes"] = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
        more["y_scales"] = torch.empty((cols + 127) // 128, rows, 4, dtype=torch.uint8, device="cuda")
        out["y_held"] = torch.empty_like(x)
    if st["checkpoint"]:
        more["ck_codes"] = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
        more["ck_scales"] = torch.empty(rows, cols // 32, dtype=torch.uint8, device="cuda")
        out["sum_held"] = torch.empty_like(x)
    moe.moe_add_rmsnorm_fwd(x, st["gain"], y, eps=EPS, residual=r, summed=s, rstd=out["rstd"], **more)
    if st["codes"]:
        moe.moe_mx_dequantize(more["y_codes"], more["y_scales"], out["y_held"], operand_scales=True)
    if st["checkpoint"]:
        moe.moe_mx_dequantize(more["ck_codes"], more["ck_scales"], out["sum_held"])
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- from the definition, in 64 bits


def _nearest(v):
    """MXFP8 of the last axis of v, in 64 bits: scale by search over the powers of two, element by
    the nearest of E4M3's values (a tie to the even code)."""
    grid = torch.arange(127, dtype=torch.uint8, device=v.device).view(torch.float8_e4m3fn).double()
    b = v.double().reshape(-1, 32)
    amax = b.abs().amax(1, keepdim=True)
    e = torch.ceil(torch.log2(amax / 448))
    e = torch.where(amax > 448 * 2.0 ** e, e + 1, e)
    e = torch.where(amax <= 448 * 2.0 ** (e - 1), e - 1, e)
    e = torch.where(amax == 0, 0, e).clamp(-127, 127)
    q = b * 2.0 ** -e
    mid = (grid[1:] + grid[:-1]) / 2
    a = q.abs().contiguous()
    low, high = torch.bucketize(a, mid, right=False), torch.bucketize(a, mid, right=True)
    at = torch.where(low % 2 == 0, low, high)  # the two differ at a tie only: the even one
    return (torch.copysign(grid[at], q) * 2.0 ** e).reshape(v.shape)


def _exact_layer(st, x):
    mx, k = st["prec"] == "mxfp8", st["k"]
    x = x.double()
    z = x @ st["Wr"].double() + (0 if st["b"] is None else st["b"].double())
    order = torch.argsort(z, dim=1, descending=True, stable=True)[:, :k]
    chosen = torch.zeros_like(z, dtype=torch.bool).scatter_(1, order, True)
    w = torch.softmax(z.masked_fill(~chosen, -math.inf), 1)
    xq = _nearest(x) if mx else x
    out = torch.zeros_like(x)
    Wg, Wu, Wd = st["W"]
    for e in range(st["E"]):
        t = chosen[:, e].nonzero()[:, 0]
        if len(t):
            g = xq[t] @ Wg[e].double()
            h = g * torch.sigmoid(g) * (xq[t] @ Wu[e].double())
            out[t] += w[t, e, None] * ((_nearest(h) if mx else h) @ Wd[e].double())
    if st["shared"]:
        Sg, Su, Sd = (s.double() for s in st["S"])
        g = x @ Sg
        out += (g * torch.sigmoid(g) * (x @ Su)) @ Sd
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "few":
        return _exact_layer(st, st["x"])
    if case["op"] == "norm_bwd":
        s = (_values(st["codes"], st["scales"]) if case["checkpoint"] else st["s"]).double()
        dy, rstd, gain = st["dy"].double(), st["rstd"].double()[:, None], st["gain"].double()
        # y_i = gain_i s_i rstd(s): its Jacobian's transpose on dy
        dot = (dy * gain * s).sum(1, keepdim=True)
        dx = rstd * gain * dy - s * rstd ** 3 * dot / case["cols"]
        if st["dsum"] is not None:
            dx = dx + st["dsum"].double()
        return {"dx": dx, "dgain": (dy * s * rstd).sum(0)}
    s = st["x"].double()
    if st["residual"] is not None:
        s = (s + st["residual"].double()).bfloat16().double()  # the stream is held in bf16
    rstd = (s.square().mean(1) + EPS).rsqrt()
    y = s * rstd[:, None] * st["gain"].double()
    if case["op"] == "block":
        return {"sum": s, "out": _exact_layer(st, y.bfloat16())}  # the layer takes bf16
    out = {"y": y, "rstd": rstd}
    if st["residual"] is not None:
        out["sum"] = s
    if case["codes"]:
        out["y_held"] = _nearest(y.bfloat16())
    if case["checkpoint"]:
        out["sum_held"] = _nearest(s)
    return out
