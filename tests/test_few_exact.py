"""The few-token layer (moe_layer_fwd_few) on inputs whose every sum is exact, so that
its outputs have to equal the formula's bit for bit: each column of H, and each of I, is
the only one that some token's output hangs on.  A bound on rounding errors over long
sums cannot see one that is left out, taken twice or read from another place; these
tests do, and the CPU part shows it for the formula with columns taken out.

Why nothing is rounded: a token's gate is 64 through one product (silu(64) is 64 in
fp32), its up values are single products of a value of four significant bits and a power
of two, MXFP8 holds both (a block of 32 has one weight, or values within 2^4 of each
other), the chosen experts weigh 1/k with k a power of two, and what an output adds up
are few such values within 2^20 of each other, rounded once to bf16.
"""
import ctypes

import numpy as np
import pytest
import torch

import dispatch_grouped_gemm_moe_amd as moe
import oracle as O
from few_reference import HALF_BF16, few_layer
from moe_inputs import LayerInputs, Workload, make_inputs
from test_few import Few, test_few_routes_as_the_router_does as routes_as_the_router_does

G = 64  # columns that a token reads at a time


def _workload(T, H, I, E, k, prec, shared):
    return Workload("exact_%d_%d_%d_%d_%d_%s_%d" % (T, H, I, E, k, prec, shared), T=T, H=H, I=I, E=E, k=k, prec=prec,
                    shared_expert=shared)


def _chosen(j, E, k):
    """The experts of the tokens of group j."""
    return [(5 * j + m) % E for m in range(k)]


def _value(c, j):
    """Four significant bits, either sign, magnitudes 0.5 to 3.75."""
    return (-1) ** ((c + j) // 3) * (1 + (c + j) % 8 / 8) * 2.0 ** (c % 3 - 1)


def _down(E, I, H):
    """Wd of every expert and of the shared one: output column c takes the I columns that c % 64 says."""
    i, c = torch.arange(I)[:, None], torch.arange(H)[None, :]
    base = torch.where(i % G == c % G, 2.0 ** (i // G % 4 + c // G % 2), 0.0)
    return torch.stack([base * 2.0 ** (e % 4) for e in range(E)] + [base * 32]).bfloat16()


def _up(rows, cols, E, block):
    """Wu: column i takes the row h with h % 64 = i % 64, times a power of two by expert and block."""
    h, i = torch.arange(rows)[:, None], torch.arange(cols)[None, :]
    on = (h % G == i % G) & (h % G != G - 1)
    return torch.stack([torch.where(on, 2.0 ** ((block(h, i) + e) % 3 - 1), 0.0) for e in range(E + 1)]).bfloat16()


class ByH:
    """Token t of round r reads columns 64 j .. 64 j + 63 of H, j = (T r + t) mod H / 64: 63 values for
    Wu and, in the last, a 1 for the gate and the router."""

    def __init__(self, T, H, I, E, k, prec, shared):
        self.w = _workload(T, H, I, E, k, prec, shared)
        self.groups, self.rounds = H // G, -(-H // G // T)
        Wu, Wd = _up(H, I, E, lambda h, i: h // G), _down(E, I, H)
        Wg = torch.zeros(E + 1, H, I, dtype=torch.bfloat16)
        Wg[:, G - 1::G] = 64
        Wr = torch.zeros(H, E)
        for j in range(self.groups):
            Wr[G * j + G - 1, _chosen(j, E, k)] = 4
        s = lambda m: m[E].contiguous() if shared else None
        self.inp = LayerInputs(self.w, torch.zeros(T, H, dtype=torch.bfloat16), Wr, None, Wg[:E].contiguous(),
                               Wu[:E].contiguous(), Wd[:E].contiguous(), s(Wg), s(Wu), s(Wd))
        self.Wu, self.Wd = Wu.double(), Wd.double()

    def group(self, t, r):
        return (self.w.T * r + t) % self.groups

    def tokens(self, r):
        x = torch.zeros(self.w.T, self.w.H)
        for t in range(self.w.T):
            j = self.group(t, r)
            x[t, G * j:G * j + G] = torch.tensor([_value(c, j) for c in range(G - 1)] + [1.0])
        return x.bfloat16()

    def up(self, x, t, j, e):
        """The one product in each of token t's up values for expert e."""
        i = torch.arange(self.w.I)
        return x[t].double()[G * j + i % G] * self.Wu[e][G * j + i % G, i]

    def want(self, r):
        """The formula's outputs, rounded to bf16."""
        w, x = self.w, self.tokens(r)
        out = torch.zeros(w.T, w.H, dtype=torch.float64)
        for t in range(w.T):
            j = self.group(t, r)
            for e in _chosen(j, w.E, w.k):
                out[t] += 64 * self.up(x, t, j, e) @ self.Wd[e] / w.k
            if w.shared_expert:
                out[t] += 64 * self.up(x, t, j, w.E) @ self.Wd[w.E]
        return out.bfloat16()  # (a sum of few bits: fp32 in between changes nothing)


class ByI(ByH):
    """Token t of round r has a gate for columns 64 j .. 64 j + 63 of I only, j = (T r + t) mod I / 64.
    Columns of H: 63 values, then a gate column for each j, then a router column for each token."""

    def __init__(self, T, H, I, E, k, prec, shared):
        self.w = _workload(T, H, I, E, k, prec, shared)
        self.groups, self.rounds = I // G, -(-I // G // T)
        assert H >= G + self.groups + T
        Wu, Wd = _up(H, I, E, lambda h, i: i // G), _down(E, I, H)
        Wu[:, G:] = 0
        Wg = torch.zeros(E + 1, H, I, dtype=torch.bfloat16)
        for j in range(self.groups):
            Wg[:, G + j, G * j:G * j + G] = 64
        Wr = torch.zeros(H, E)
        for t in range(T):
            Wr[G + self.groups + t, _chosen(t, E, k)] = 4
        s = lambda m: m[E].contiguous() if shared else None
        self.inp = LayerInputs(self.w, torch.zeros(T, H, dtype=torch.bfloat16), Wr, None, Wg[:E].contiguous(),
                               Wu[:E].contiguous(), Wd[:E].contiguous(), s(Wg), s(Wu), s(Wd))
        self.Wu, self.Wd = Wu.double(), Wd.double()

    def tokens(self, r):
        x = torch.zeros(self.w.T, self.w.H)
        for t in range(self.w.T):
            x[t, :G - 1] = torch.tensor([_value(c, t) for c in range(G - 1)])
            x[t, G + self.group(t, r)] = 1
            x[t, G + self.groups + t] = 1
        return x.bfloat16()

    def want(self, r):
        w, x = self.w, self.tokens(r)
        out = torch.zeros(w.T, w.H, dtype=torch.float64)
        for t in range(w.T):
            at = torch.arange(G * self.group(t, r), G * self.group(t, r) + G)
            for e in _chosen(t, w.E, w.k) + ([w.E] if w.shared_expert else []):
                u = x[t].double()[at % G] * self.Wu[e][at % G, at]
                out[t] += 64 * u @ self.Wd[e][at] * (1 if e == w.E else 1 / w.k)
        return out.bfloat16()


# (T, H, I, E, k): H split over workgroups and not, rows of an odd multiple of 64 columns, more than one and
# more than two slabs of the router, experts of up to 8, 16, 32 and 64 rows
BY_H = [(7, 8256, 64, 1, 1), (4, 4160, 192, 6, 2), (50, 6208, 128, 2, 2), (1, 3136, 64, 32, 4), (7, 8256, 64, 8, 2),
        (5, 16448, 64, 7, 4), (11, 8256, 64, 65, 8), (13, 832, 64, 2, 2), (30, 1984, 128, 2, 2), (64, 4160, 64, 3, 1),
        (64, 2112, 320, 4, 4)]
# I in parts over waves and workgroups
BY_I = [(9, 256, 1984, 8, 4), (9, 256, 1984, 40, 8), (16, 256, 2048, 64, 16), (1, 1024, 448, 32, 8),
        (7, 448, 64, 256, 16), (3, 2048, 960, 16, 4), (2, 4224, 704, 9, 4), (16, 192, 1984, 2, 2), (20, 192, 1984, 2, 2),
        (33, 256, 1984, 8, 4), (64, 192, 1088, 4, 4), (64, 192, 1984, 1, 1)]
ALL = [(ByH, s) for s in BY_H] + [(ByI, s) for s in BY_I]
IDS = ["%s-%s" % (c.__name__, "-".join(map(str, s))) for c, s in ALL]


# ------------------------------------------------------------------ the formula itself (no GPU)

@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
@pytest.mark.parametrize("by,shape", [(ByH, BY_H[1]), (ByH, BY_H[3]), (ByH, BY_H[0]), (ByH, BY_H[2]), (ByI, BY_I[0])])
def test_a_column_left_out_changes_the_formulas_outputs(by, shape, prec, shared):
    case = by(*shape, prec, shared)
    inp, T = case.inp, shape[0]

    def layer(r):
        inp.x = case.tokens(r)
        return torch.from_numpy(few_layer(inp, T)[0]).bfloat16()

    for j in {0, case.groups // 2, case.groups - 1}:
        r, t = divmod(j, T)
        want = case.want(r)
        assert torch.equal(layer(r), want)  # the 64-bit layer rounds nothing either
        axis = 1 if by is ByH else 2
        kept = [m.clone() for m in (inp.Wg, inp.Wu, inp.Wd)]
        for m, a in ((inp.Wg, axis), (inp.Wu, axis)) if by is ByH else ((inp.Wd, 1),):
            m.narrow(a, G * j, G).zero_()
        assert not torch.equal(layer(r)[t], want[t])
        for m, old in zip((inp.Wg, inp.Wu, inp.Wd), kept):
            m.copy_(old)


@pytest.mark.parametrize("E,k", [(8, 3), (7, 2)])
def test_the_routers_second_slab_decides(E, k):
    # the inputs of the GPU test below: without the columns past 8192 every token's weights are others
    inp = _slab_inputs(5, 8256, E, k)
    x = inp.x.float().numpy()
    _, idx, gw = O.route(x, inp.Wr, None, k)
    x[:, 8192:] = 0
    _, idx2, gw2 = O.route(x, inp.Wr, None, k)
    assert ((idx != idx2).any(1) | (np.abs(gw - gw2).max(1) > 0.01)).all()


def _slab_inputs(T, H, E, k):
    inp = make_inputs(Workload("slab_%d_%d_%d_%d" % (T, H, E, k), T=T, H=H, I=64, E=E, k=k, stream=9800 + E))
    inp.Wr[H // 8192 * 8192:] *= 10  # the 64 columns of the last slab weigh as much as all the others
    return inp


# ------------------------------------------------------------------ GPU

def _splits(name, *args):
    """What the launch makes of a product: an internal function of the library."""
    f = getattr(moe.lib(), name)
    f.restype, f.argtypes = ctypes.c_int, [ctypes.c_int64 if n == "l" else ctypes.c_int for n in name[-2:]]
    return f(*args)


def _gate_up_splits(T, H, I, E, k, prec, shared):
    return _splits("_ZN3moe18few_gate_up_splitsEli", (min(E, T * k) + shared) * (I // 32),
                   H * (1 if prec == "mxfp8" and not shared else 2))


def _down_splits(T, H, I, E, k, prec, shared):
    return _splits("_ZN3moe17few_down16_splitsEil", H, (min(E, T * k) + shared) * 16 * I * (1 if prec == "mxfp8" else 2)
                   // 1024)


def test_the_cases_take_the_products_in_parts():
    for prec in ("bf16", "mxfp8"):
        for shared in (False, True):
            gate_up = [_gate_up_splits(*s, prec, shared) for s in BY_H]
            assert min(gate_up) == 1 and max(gate_up) >= 5 and len(set(gate_up)) >= 3, gate_up
            down = [_down_splits(*s, prec, shared) for s in BY_I if s[0] <= 16]
            assert min(down) == 1 and max(down) == 8 and len(set(down)) >= 3, down


@pytest.mark.gpu
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
@pytest.mark.parametrize("by,shape", ALL, ids=IDS)
def test_few_takes_every_column_once(gpu_lib, by, shape, prec, shared):
    case = by(*shape, prec, shared)
    few = Few(case.w, case.inp)
    for r in range(case.rounds):
        got, want = few(case.tokens(r).cuda()).cpu(), case.want(r)
        wrong = (got != want).nonzero()
        assert len(wrong) == 0, "round %d: %d outputs, the first at %s: %s for %s" % (
            r, len(wrong), wrong[0].tolist(), got[tuple(wrong[0])].item(), want[tuple(wrong[0])].item())


@pytest.mark.gpu
@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
@pytest.mark.parametrize("shape", [(5, 8256, 64, 8, 3), (6, 16448, 64, 7, 2), (3, 8256, 64, 67, 5), (9, 16448, 64, 12, 4)],
                         ids=lambda s: "-".join(map(str, s)))
def test_few_routes_as_the_router_does_past_a_slab(gpu_lib, shape, prec):
    routes_as_the_router_does(gpu_lib, shape, prec)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,E,k", [(5, 8256, 8, 3), (5, 8256, 7, 2), (6, 16448, 12, 4), (3, 16448, 67, 5)])
def test_few_router_by_its_last_slab(gpu_lib, T, H, E, k):
    # expert e's output is 1 in column e (silu(64) / 64 is 1): the layer's are the routing weights
    inp = _slab_inputs(T, H, E, k)
    inp.x[:, 0] = 1
    for m in (inp.Wg, inp.Wu, inp.Wd):
        m.zero_()
    inp.Wg[:, 0, 0], inp.Wu[:, 0, 0] = 64, 1 / 64
    for e in range(E):
        inp.Wd[e, 0, e] = 1
    _, idx, gw = O.route(inp.x.float().numpy(), inp.Wr, None, k)
    few = Few(inp.w, inp)
    want = torch.zeros(T, H).scatter_(1, torch.from_numpy(idx.astype(np.int64)), torch.from_numpy(gw.astype(np.float32)))
    # (the softmax's exp is the device's: 2^-19 relative, besides bf16's half step)
    assert ((few().cpu().float() - want).abs() <= want * (HALF_BF16 + 2.0 ** -19)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 9, 20, 40])
@pytest.mark.parametrize("I", [64, 192, 1984])
def test_few_mxfp8_down_product_keeps_what_the_matrix_instruction_keeps(gpu_lib, T, I):
    """The scaled matrix instruction adds up eight neighbouring products on one exponent: what lies
    below 2^-13 of the largest is cut off.  Everything else is fp32.  So a sum is off by at most 7 2^-13
    of the sum of the groups' largest magnitudes, and n 2^-23 of the whole.  Here each group has a large
    product, which the next group's takes away again, and seven of 2^-14 to 2^-11 of it."""
    w = _workload(T, 128, I, 2, 2, "mxfp8", False)
    x, Wg, Wu = torch.zeros(T, 128), torch.zeros(2, 128, I), torch.zeros(2, 128, I)
    x[:, 0] = 1
    x[:, 1] = 2.0 ** (torch.arange(T) % 3)
    Wg[:, 0] = 64
    i = torch.arange(I)
    Wu[:, 1] = torch.where(i % 8 == 0, 1.0, 2.0 ** -6)  # h: 64 or 1, times the token's
    c = torch.arange(128)[None, :]
    small = 2.0 ** -(5 + c % 4).float() * torch.where((i[:, None] + c) % 5 < 3, 1.0, -1.0)
    Wd = torch.where(i[:, None] % 8 == 0, torch.where(i[:, None] % 16 == 0, 1.0, -1.0), small).expand(2, I, 128)
    inp = LayerInputs(w, x.bfloat16(), torch.zeros(128, 2), None, *(m.bfloat16().contiguous() for m in (Wg, Wu, Wd)))
    h = (64 * inp.x[:, 1:2].double()) * inp.Wu[0, 1].double()
    W = inp.Wd[0].double()
    # MXFP8 holds h (64 or 1 of a block's scale) and the weights (1 to 2^-8) exactly
    want = h @ W
    mag = h.abs() @ W.abs()
    largest = (h[:, ::8].abs() @ W[::8].abs())
    got = Few(w, inp)().double().cpu()
    bound = 7 * 2.0 ** -13 * largest + I * 2.0 ** -23 * mag
    assert ((got - want).abs() <= bound + HALF_BF16 * (want.abs() + bound)).all()
