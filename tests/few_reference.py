"""The few-token layer in 64 bits, with a bound on how far an implementation that
rounds where the library's documentation says it rounds can be from it.

What is rounded: the router's fp32 logits (the oracle's fixed order gives them
bit for bit) and softmax; bf16 precision holds h in two bf16 parts, MXFP8 quantises x
(exactly defined) and h; every sum is fp32; the output is bf16.  The bound adds
what each of these can move the output by, element by element:

* a sum of n products in fp32: n 2^-23 times the sum of their magnitudes (twice
  the textbook n 2^-24, as a matrix instruction may truncate where it aligns);
* silu(g) u for errors dg, du: |silu'| <= 1.1, plus 2^-20 relative for exp and
  the division;
* h to two bf16 parts, the first cut off: half a step of a step, 2^-15 relative;
* h to MXFP8: the scale and the code of h +- dh, the farthest of the cases;
* the gate weight: 2^-19 relative (exp of a difference of logits);
* the output: half a bf16 step, 2^-8 relative.
"""
import numpy as np

import oracle as O

F32 = 2.0 ** -23
HALF_BF16 = 2.0 ** -8


def _point(v, e):
    """v held in E4M3 times 2^e (round to nearest even, saturating), in 64 bits."""
    q = v * np.ldexp(1.0, -e)[:, None]
    _, p = np.frexp(q)
    step = np.ldexp(1.0, np.maximum(p, -5) - 4)
    q = np.clip(np.round(q / step) * step, -448, 448)
    return q * np.ldexp(1.0, e)[:, None]


def few_layer(inp, T):
    """(out, bound) [T, H] of the first T tokens of `inp`."""
    w = inp.w
    mx = w.prec == "mxfp8"
    x = O.as_f64(inp.x)[:T]
    _, idx, gw = O.route(x.astype(np.float32), inp.Wr, inp.bias, w.k)
    xq = O.mx_roundtrip(x, axis=1) if mx else x
    H, I = w.H, w.I
    out, bound = np.zeros((T, H)), np.zeros((T, H))

    def expert(rows, a, Wg, Wu, Wd, wt, quant):
        g, u = a @ Wg, a @ Wu
        dg, du = H * F32 * (np.abs(a) @ np.abs(Wg)), H * F32 * (np.abs(a) @ np.abs(Wu))
        s = g / (1 + np.exp(np.minimum(-g, 700.0)))
        h = s * u
        dh = 1.1 * dg * (np.abs(u) + du) + np.abs(s) * du + 2.0 ** -20 * np.abs(h)
        if quant:
            b, d = h.reshape(-1, 32), dh.reshape(-1, 32)
            e0 = O.e8m0_scale_exponent(np.abs(b).max(1))
            ref = _point(b, e0)
            err = np.zeros_like(b)
            for e in (O.e8m0_scale_exponent(np.maximum(np.abs(b) - d, 0).max(1)),
                      O.e8m0_scale_exponent((np.abs(b) + d).max(1))):
                for sg in (-1, 1):
                    err = np.maximum(err, np.abs(_point(b + sg * d, e) - ref))
            h, dh = ref.reshape(h.shape), err.reshape(h.shape)
        else:
            dh = dh + 2 * HALF_BF16 ** 2 * (np.abs(h) + dh)
        y = h @ Wd
        mag = np.abs(h) @ np.abs(Wd)
        dy = dh @ np.abs(Wd) + I * F32 * (mag + dh @ np.abs(Wd))
        out[rows] += wt * y
        bound[rows] += np.abs(wt) * (dy + 2.0 ** -19 * np.abs(y)) + (w.k + 2) * F32 * np.abs(wt * y)

    for e in range(w.E):
        t, j = np.nonzero(idx == e)
        if not t.size:
            continue
        W = [O.as_f64(m[e]) for m in (inp.Wg, inp.Wu, inp.Wd)]
        if mx:
            W = [O.mx_roundtrip(m, axis=0) for m in W]
        expert(t, xq[t], *W, gw[t, j][:, None].astype(np.float64), mx)
    if w.shared_expert:
        expert(np.arange(T), x, *[O.as_f64(m) for m in (inp.Wsg, inp.Wsu, inp.Wsd)], np.ones((T, 1)), False)
    return out, bound + HALF_BF16 * (np.abs(out) + bound) + 1e-38
