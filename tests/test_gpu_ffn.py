"""The experts' block, its gradient, combine's gradient and 8-bit products on the GPU
against 64 bits, at the sizes and layouts where they can go wrong."""
import pytest
import torch

import combine_ep_get_amd as ep
from tests import ffn_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
NAN = float("nan")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF)


def routing(g, N, K, E, skew=0.0, drop=0.0):
    likes = torch.randn((E,), generator=g, device="cuda") * skew
    noise = -torch.log(-torch.log(torch.rand((N, E), generator=g, device="cuda")
                                  .clamp(1e-6, 1 - 1e-6)))
    idx = torch.sort(likes + noise, dim=1, descending=True)[1][:, :K]
    gone = torch.rand((N, K), generator=g, device="cuda") < drop
    return torch.where(gone, torch.full_like(idx, -1), idx).to(torch.int32).contiguous()


def scatter(cap, cols, at, rows, fill=NAN):
    """A buffer whose rows `at` are `rows`, all others `fill`."""
    out = torch.full((cap, cols), fill, dtype=rows.dtype, device="cuda")
    out[at] = rows
    return out


class Case:
    """A layout, x with NaN where no row is, and weights."""

    def __init__(self, seed, N, K, E, A, H, I, R=1, skew=0.5, drop=0.1, ll=0, int8=False):
        g = self.g = gen(seed)
        self.H, self.I = H, I
        if E == 0:
            self.layout, self.cap, lead = None, N, ()
        else:
            self.idx = routing(g, N, K, E, skew, drop)
            lead = (E,)
            if ll:
                xs, w = normal(g, N, H), torch.ones((N, K), device="cuda")
                self.layout, _ = ep.ll_dispatch(xs, self.idx, w, E, R, ll)
            else:
                self.layout = ep.get_layout(self.idx, E, R, A)
            self.cap = self.layout.capacity
        self.where = [(e, s.cuda()) for e, s in ref.slots_of(self.layout, self.cap)]
        self.at = torch.cat([s for _, s in self.where])
        self.rest = torch.ones((self.cap,), dtype=torch.bool, device="cuda")
        self.rest[self.at] = False
        self.x = self.rows(H)
        if int8:
            self.w13 = ep.Int8Weight.from_weight(normal(g, *lead, 2 * I, H, scale=H ** -0.5))
            self.w2 = ep.Int8Weight.from_weight(normal(g, *lead, H, I, scale=I ** -0.5))
        else:
            self.w13 = normal(g, *lead, 2 * I, H, scale=H ** -0.5)
            self.w2 = normal(g, *lead, H, I, scale=I ** -0.5)

    def rows(self, cols):
        return scatter(self.cap, cols, self.at, normal(self.g, len(self.at), cols))

    def untouched(self, t, value=7.0):
        assert bool((t[self.rest] == value).all()), "a slot without a row was written"

    def full(self, cols, value=7.0):
        return torch.full((self.cap, cols), value, dtype=BF, device="cuda")


SHAPES = [
    dict(N=1, K=1, E=1, A=1, H=8, I=8, drop=0),                        # one of everything
    dict(N=1, K=2, E=4, A=1, H=72, I=40),
    dict(N=37, K=2, E=5, A=4, H=136, I=72),                            # ends inside a step
    dict(N=128, K=2, E=16, A=1, H=256, I=128),                         # the tiny workload
    dict(N=300, K=3, E=7, A=16, H=264, I=200, skew=2.0),               # uneven experts
    dict(N=600, K=2, E=3, A=128, H=512, I=264, drop=0.4),              # several row tiles
    dict(N=64, K=1, E=64, A=1, H=64, I=64, skew=3.0),                  # many empty experts
    dict(N=5, K=1, E=1024, A=1, H=16, I=16),                           # most experts
    dict(N=256, K=1, E=0, A=1, H=320, I=256),                          # plain, a whole tile
    dict(N=257, K=1, E=0, A=1, H=1000, I=344),                         # plain, one row over
    dict(N=1, K=1, E=0, A=1, H=2048, I=1024),                          # plain, one token
    dict(N=2100, K=1, E=0, A=1, H=128, I=64),                          # more than 8 row tiles
]


def ident(c):
    return "-".join(f"{k}{v}" for k, v in c.items())


def check_ffn(c, y, gu=None):
    for e, s in c.where:
        if len(s) == 0:
            continue
        want, bound, wgu, bgu = ref.ffn(c.x[s].double(), ref.pick(c.w13, e), ref.pick(c.w2, e))
        ref.check(y[s], want, bound, f"y of expert {e}")
        if gu is not None:
            ref.check(gu[s], wgu, bgu, f"gate_up of expert {e}")


@pytest.mark.parametrize("shape", SHAPES, ids=ident)
def test_forward(shape):
    c = Case(1, **shape)
    y, gu = c.full(c.H), c.full(2 * c.I)
    ep.expert_ffn(c.x, c.w13, c.w2, layout=c.layout, out=y, gate_up=gu)
    check_ffn(c, y, gu)
    c.untouched(y)
    c.untouched(gu)
    again = ep.expert_ffn(c.x, c.w13, c.w2, layout=c.layout)       # no gate_up, its own memory
    assert torch.equal(again[c.at], y[c.at])


@pytest.mark.parametrize("shape", [
    dict(N=8, K=2, E=4, A=1, H=64, I=32, R=2, ll=4),
    dict(N=48, K=3, E=12, A=1, H=272, I=144, R=4, ll=12),
    dict(N=256, K=8, E=32, A=1, H=512, I=256, R=8, ll=32),
    dict(N=600, K=2, E=2, A=1, H=128, I=64, R=2, ll=300, drop=0),      # rows of both sources
], ids=ident)
@pytest.mark.parametrize("int8", [False, True])
def test_forward_low_latency(shape, int8):
    c = Case(2, int8=int8, **shape)
    y = ep.expert_ffn(c.x, c.w13, c.w2, layout=c.layout, out=c.full(c.H))
    c.untouched(y)
    if int8:
        check_int8_ffn(c, y)
    else:
        check_ffn(c, y)


@pytest.mark.parametrize("shape", SHAPES, ids=ident)
def test_backward(shape):
    c = Case(3, **shape)
    gu, dy = c.rows(2 * c.I), c.rows(c.H)
    dx = c.full(c.H)
    dw13, dw2 = torch.full_like(c.w13, NAN), torch.full_like(c.w2, NAN)
    out = ep.expert_ffn_backward(dy, c.x, gu, c.w13, c.w2, layout=c.layout, out=(dx, dw13, dw2))
    assert all(a is b for a, b in zip(out, (dx, dw13, dw2)))
    c.untouched(dx)
    for e, s in c.where:
        g13, g2 = (dw13, dw2) if e is None else (dw13[e], dw2[e])
        if len(s) == 0:
            assert not bool(g13.any()) and not bool(g2.any()), f"expert {e} has no rows"
            continue
        (wx, bx), (w13, b13), (w2, b2) = ref.ffn_grad(
            dy[s].double(), c.x[s].double(), gu[s].double(), ref.pick(c.w13, e),
            ref.pick(c.w2, e))
        ref.check(dx[s], wx, bx, f"dx of expert {e}")
        ref.check(g13, w13, b13, f"dw13 of expert {e}")
        ref.check(g2, w2, b2, f"dw2 of expert {e}")
    again = ep.expert_ffn_backward(dy, c.x, gu, c.w13, c.w2, layout=c.layout)
    assert torch.equal(again[0][c.at], dx[c.at])
    assert torch.equal(again[1], dw13) and torch.equal(again[2], dw2)


def test_backward_without_rows():
    w13, w2 = normal(gen(4), 2, 32, 16), normal(gen(4), 2, 16, 16)
    lay = ep.get_layout(torch.empty((0, 1), dtype=torch.int32, device="cuda"), 2, 1)
    e = torch.empty((0, 16), dtype=BF, device="cuda")
    gu = torch.empty((0, 32), dtype=BF, device="cuda")
    out = (e.clone(), torch.full_like(w13, NAN), torch.full_like(w2, NAN))
    ep.expert_ffn_backward(e, e, gu, w13, w2, layout=lay, out=out)
    assert not bool(out[1].any()) and not bool(out[2].any())
    assert ep.expert_ffn(e, w13, w2, layout=lay).shape == (0, 16)
    none = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")        # rows, but nobody's
    lay = ep.get_layout(none, 2, 1)
    x = torch.full((lay.capacity, 16), NAN, dtype=BF, device="cuda")
    gu = torch.full((lay.capacity, 32), NAN, dtype=BF, device="cuda")
    dx, dw13, dw2 = ep.expert_ffn_backward(x, x, gu, w13, w2, layout=lay,
                                           out=(x.clone(), *out[1:]))
    assert bool(dx.isnan().all()) and not bool(dw13.any()) and not bool(dw2.any())


def test_values_stay_in_their_row():
    """An infinity or NaN in a row of x reaches that row of y only, and a huge gate is no NaN."""
    c = Case(5, N=70, K=1, E=0, A=1, H=64, I=32)
    clean = ep.expert_ffn(c.x, c.w13, c.w2)
    x = c.x.clone()
    x[3, 5], x[41, 0] = NAN, float("inf")
    y = ep.expert_ffn(x, c.w13, c.w2)
    assert bool(y[3].isnan().all()) and not bool(y[41].isfinite().all())
    keep = torch.ones(70, dtype=torch.bool, device="cuda")
    keep[[3, 41]] = False
    assert torch.equal(y[keep], clean[keep])
    big = torch.full((2, 64), 1000.0, dtype=BF, device="cuda")
    big[1] = -1000.0
    w13 = torch.ones((64, 64), dtype=BF, device="cuda")
    y = ep.expert_ffn(big, w13, c.w2)
    want = ref.ffn(big.double(), w13.double(), c.w2.double())
    ref.check(y, want[0], want[1], "saturated gates")
    gu = torch.full((2, 64), 200.0, dtype=BF, device="cuda")
    gu[1] = -200.0
    dy = torch.ones((2, 64), dtype=BF, device="cuda")
    for t in ep.expert_ffn_backward(dy, big, gu, w13, c.w2):
        assert bool(t.isfinite().all())


# ------------------------------------------------------------------ 8-bit integers
def check_int8_ffn(c, y):
    """A code of h is off by at most one where its rounding to bf16 or to an integer is on
    an edge, so a value of y by at most a step of h's scale times the weights; over a whole
    matrix such edges are rare, and what is left is y's own rounding."""
    got, want = [], []
    for e, s in c.where:
        if len(s) == 0:
            continue
        q13, s13 = (t if e is None else t[e] for t in (c.w13.codes, c.w13.scales))
        q2, s2 = (t if e is None else t[e] for t in (c.w2.codes, c.w2.scales))
        qx, sx = ref.quantize(c.x[s])
        gu = (qx @ q13.double().t()) * sx.double()[:, None] * s13.double()
        h = (ref.silu_parts(gu[:, :c.I])[1] * gu[:, c.I:]).to(BF)
        qh, sh = ref.quantize(h)
        w = (qh @ q2.double().t()) * sh.double()[:, None] * s2.double()
        slack = sh.double()[:, None] * q2.double().abs().sum(dim=1) * s2.double()
        ref.check(y[s], w, slack + 2 * ref.BF16 * (w.abs() + slack), f"y of expert {e}")
        got.append(y[s].double())
        want.append(w)
    got, want = torch.cat(got), torch.cat(want)
    if got.numel() >= 4096:
        assert float((got - want).norm() / want.norm()) < ref.BF16


@pytest.mark.parametrize("shape", [
    dict(N=1, K=1, E=1, A=1, H=16, I=16, drop=0),
    dict(N=37, K=2, E=5, A=4, H=144, I=80),
    dict(N=300, K=3, E=7, A=16, H=272, I=208, skew=2.0),
    dict(N=700, K=2, E=3, A=128, H=512, I=272, drop=0.4),
    dict(N=257, K=1, E=0, A=1, H=1008, I=352),
    dict(N=1, K=1, E=0, A=1, H=2048, I=1024),
], ids=ident)
def test_int8_ffn(shape):
    c = Case(6, int8=True, **shape)
    y = ep.expert_ffn(c.x, c.w13, c.w2, layout=c.layout, out=c.full(c.H))
    check_int8_ffn(c, y)
    c.untouched(y)


@pytest.mark.parametrize("cols", [16, 128, 2048, 2064, 7168, 8192, 8208, 65536])
def test_quantize(cols):
    g = gen(7)
    n = 9 if cols > 8000 else 300
    x = normal(g, n, cols)
    x[1] = 0
    x[2] = torch.where(x[2] > 0, 1.0, -1.0)                # every value an extreme
    x[3] *= 1e30
    x[4] = (x[4].float() * 1e-38).to(BF)                   # subnormal and tiny
    x[5] = 0
    x[5, 3] = 2.0 ** -133                                  # the least bf16
    x[6] = ((torch.arange(cols, device="cuda") % 255 - 127) / 2).to(BF)     # halves: ties
    x[6, 0] = 127.0
    x[7] = x[6] * 0.75                                     # quotients that are halves again
    codes, scales = ep.quantize_int8(x)
    q, s = ref.quantize(x)
    assert torch.equal(scales, s)
    assert torch.equal(codes.double(), q)


def test_quantize_every_pair():
    """All bf16 magnitudes of a binade above all maxima of another: each code is the nearest
    integer of the exact quotient (integers: |2 x 2^k - (2 q) s| <= s, ties even)."""
    m = torch.arange(128, device="cuda").float()
    top = (1 + m / 128) * 2.0 ** 6                         # maxima 64 .. 127.5
    v = torch.cat([(1 + m / 128) * 2.0 ** e for e in range(-2, 7)])
    x = torch.zeros((128, 1 + v.numel() + 15), device="cuda")
    x = x[:, :(1 + v.numel() + 15) // 16 * 16]
    x[:, 0] = top
    n = x.shape[1] - 1
    x[:, 1:] = torch.minimum(torch.cat([v, v])[:n][None], top[:, None])
    x[:, 2::2] *= -1
    x = x.to(BF)
    codes, scales = ep.quantize_int8(x)
    q, s = ref.quantize(x)
    assert torch.equal(scales, s) and torch.equal(codes.double(), q)


def test_quantize_non_finite():
    x = normal(gen(8), 4, 64)
    x[1, 7], x[2, 63] = float("inf"), NAN
    codes, scales = ep.quantize_int8(x)
    assert scales.isnan().tolist() == [False, True, True, False]
    assert not bool(codes[1:3].any())
    w = ep.Int8Weight.from_weight(normal(gen(9), 24, 64))
    y = ep.int8_linear(x, w)
    assert bool(y[1:3].isnan().all()) and bool(y[[0, 3]].isfinite().all())
    assert ep.quantize_int8(x[:0])[0].shape == (0, 64)


INT8 = [
    dict(N=1, E=0, C=16, O=1), dict(N=1, E=0, C=7168, O=100), dict(N=3, E=0, C=48, O=7),
    dict(N=33, E=0, C=2000, O=1237), dict(N=130, E=0, C=144, O=257),
    dict(N=700, E=0, C=1024, O=512), dict(N=64, E=9, C=208, O=131),
    dict(N=900, E=4, C=512, O=300), dict(N=40, E=300, C=32, O=33),
    dict(N=17, E=0, C=65536, O=40), dict(N=16, E=0, C=256, O=70001),
]


@pytest.mark.parametrize("c", INT8, ids=ident)
@pytest.mark.parametrize("given", [False, True], ids=["bf16", "codes"])
def test_int8_linear(c, given):
    g = gen(10)
    N, E, C, O = c["N"], c["E"], c["C"], c["O"]
    lay, cap, lead = None, N, ()
    if E:
        K = min(3, E)
        lay = ep.get_layout(routing(g, N, K, E, 1.0, 0.2), E, 1, 8)
        cap, lead = lay.capacity, (E,)
    codes = torch.randint(-128, 128, (*lead, O, C), generator=g, device="cuda").to(torch.int8)
    scales = torch.rand((*lead, O), generator=g, device="cuda") + 0.1
    w = ep.Int8Weight(codes, scales)
    where = [(e, s.cuda()) for e, s in ref.slots_of(lay, cap)]
    at = torch.cat([s for _, s in where])
    x = scatter(cap, C, at, normal(g, len(at), C))
    y = torch.full((cap, O), 7.0, dtype=BF, device="cuda")
    if given:
        q = torch.randint(-128, 128, (cap, C), generator=g, device="cuda").to(torch.int8)
        sx = torch.rand((cap,), generator=g, device="cuda") + 0.1
        ep.int8_linear(q, w, layout=lay, x_scales=sx, out=y)
    else:
        ep.int8_linear(x, w, layout=lay, out=y)
    for e, s in where:
        if len(s) == 0:
            continue
        qx, ss = (q[s].double(), sx[s]) if given else ref.quantize(x[s])
        sums = qx @ (codes if e is None else codes[e]).double().t()     # exact: below 2^53
        want = sums * ss.double()[:, None] * (scales if e is None else scales[e]).double()
        # one rounding to bf16, and the sum's, both products' and their order's in float32
        ref.check(y[s], want, (ref.BF16 + 4 * ref.F32) * want.abs(), f"y of expert {e}")
    rest = torch.ones((cap,), dtype=torch.bool, device="cuda")
    rest[at] = False
    assert bool((y[rest] == 7.0).all())


# ------------------------------------------------------------------ combine's gradient
@pytest.mark.parametrize("c", [
    dict(N=1, K=1, E=1, A=1, H=8), dict(N=5, K=3, E=4, A=1, H=72),
    dict(N=128, K=2, E=16, A=4, H=256), dict(N=33, K=8, E=32, A=16, H=7168),
    dict(N=19, K=9, E=12, A=1, H=2056), dict(N=7, K=32, E=40, A=1, H=1032),
], ids=ident)
@pytest.mark.parametrize("drop", [0.0, 0.5, 1.0])
def test_combine_backward(c, drop):
    g = gen(11)
    N, K, E, H = c["N"], c["K"], c["E"], c["H"]
    idx = routing(g, N, K, E, 0.5, drop)
    if K > 1:
        idx[0, 1] = idx[0, 0]                              # one expert twice: two slots
    lay = ep.get_layout(idx, E, 1, c["A"])
    cap = lay.capacity
    slot = lay.slot_of.long()
    used = slot[slot >= 0]
    eo = scatter(cap, H, used, normal(g, len(used), H))
    dy, wts = normal(g, N, H), torch.randn((N, K), generator=g, device="cuda")
    deo = torch.full((cap, H), 7.0, dtype=BF, device="cuda")
    dw = torch.full((N, K), NAN, device="cuda")
    ep.combine_backward(dy, eo, lay, wts, out=(deo, dw))
    t = torch.arange(N, device="cuda")[:, None].expand(N, K)[slot >= 0]
    want = wts[slot >= 0].double()[:, None] * dy[t].double()
    ref.check(deo[used], want, (ref.BF16 + ref.F32) * want.abs() * (1 + ref.BF16), "d_expert_out")
    rest = torch.ones((cap,), dtype=torch.bool, device="cuda")
    rest[used] = False
    assert bool((deo[rest] == 7.0).all())
    o = eo[used].double()
    bound = H * ref.F32 * (o.abs() * dy[t].double().abs()).sum(dim=1)
    ref.check(dw[slot >= 0], (o * dy[t].double()).sum(dim=1), bound, "d_topk_weights")
    assert not bool(dw[slot < 0].any())
    inplace = eo.clone()                                   # the gradient over its operand
    _, dw2 = ep.combine_backward(dy, inplace, lay, wts, out=(inplace, torch.empty_like(dw)))
    assert torch.equal(inplace[used], deo[used]) and torch.equal(dw, dw2)


def test_combine_backward_low_latency():
    g = gen(12)
    N, K, E, R, M, H = 64, 4, 16, 4, 16, 512
    idx = routing(g, N, K, E, 0.5, 0.2)
    wts = torch.rand((N, K), generator=g, device="cuda")
    lay, (rx, _, _, _) = ep.ll_dispatch(normal(g, N, H), idx, wts, E, R, M)
    slot = lay.slot_of.long()
    dy = normal(g, N, H)
    eo = torch.randn(rx.shape, generator=g, device="cuda").to(BF)
    deo, dw = ep.combine_backward(dy, eo, lay, wts)
    t, k = (slot >= 0).nonzero().t()
    want = wts[t, k].double()[:, None] * dy[t].double()
    ref.check(deo[slot[t, k]], want, (ref.BF16 + 2 * ref.F32) * want.abs(), "d_expert_out")
    o = eo[slot[t, k]].double() * dy[t].double()
    ref.check(dw[t, k], o.sum(dim=1), H * ref.F32 * o.abs().sum(dim=1), "d_topk_weights")


# ------------------------------------------------------------------ a run of them
def test_training_step():
    """dispatch, block, combine and back: the gradients of x, the gate weights and the
    experts' weights are those of the whole layer in 64 bits."""
    g = gen(13)
    N, K, E, H, I, A = 96, 3, 6, 128, 72, 8
    idx = routing(g, N, K, E, 0.5, 0.1)
    x, wts = normal(g, N, H), torch.rand((N, K), generator=g, device="cuda")
    w13, w2 = normal(g, E, 2 * I, H, scale=H ** -0.5), normal(g, E, H, I, scale=I ** -0.5)
    lay = ep.get_layout(idx, E, 1, A)
    rx, _, _, _ = ep.dispatch(x, wts, lay)
    gu = torch.empty((lay.capacity, 2 * I), dtype=BF, device="cuda")
    eo = ep.expert_ffn(rx, w13, w2, layout=lay, gate_up=gu)
    y = ep.combine(eo, lay, wts)
    dy = normal(g, N, H)
    deo, dwts = ep.combine_backward(dy, eo, lay, wts)
    drx, dw13, dw2 = ep.expert_ffn_backward(deo, rx, gu, w13, w2, layout=lay)
    dx = ep.combine(drx, lay, torch.ones_like(wts))

    # the same in 64 bits by torch's own differentiation, on the CPU
    leaves = [t.double().cpu().requires_grad_() for t in (x, wts, w13, w2)]
    X, W, A13, A2 = leaves
    out = torch.zeros((N, H), dtype=torch.float64)
    for e in range(E):
        t, k = (idx.cpu() == e).nonzero().t()
        both = X[t] @ A13[e].t()
        h = torch.nn.functional.silu(both[:, :I]) * both[:, I:]
        out = out.index_add(0, t, W[t, k][:, None] * (h @ A2[e].t()))
    out.backward(dy.double().cpu())
    for got, want, what in ((y, out.detach(), "y"), (dx, X.grad, "dx"), (dwts, W.grad, "dwts"),
                            (dw13, A13.grad, "dw13"), (dw2, A2.grad, "dw2")):
        err = (got.double().cpu() - want).norm() / want.norm()
        # at most five roundings to bf16 follow one another (rx none; gu, h, eo or deo, dgu,
        # the gradient itself), each at most 2^-8 of its value
        assert float(err) < 5 * ref.BF16, (what, float(err))


def test_decode_step_low_latency():
    """ll_dispatch, the block on the sub-blocks, combine: as the layer for a few tokens."""
    g = gen(14)
    N, K, E, R, H, I = 32, 4, 16, 4, 256, 128
    idx = routing(g, N, K, E, 0.5, 0.1)
    x, wts = normal(g, N, H), torch.rand((N, K), generator=g, device="cuda")
    w13, w2 = normal(g, E, 2 * I, H, scale=H ** -0.5), normal(g, E, H, I, scale=I ** -0.5)
    lay, (rx, _, _, _) = ep.ll_dispatch(x, idx, wts, E, R, N // R)
    y = ep.combine(ep.expert_ffn(rx, w13, w2, layout=lay), lay, wts)
    other = ep.moe_layer(x, idx, wts, w13, w2)
    assert float((y.double() - other.double()).norm() / other.double().norm()) < 4 * ref.BF16


@pytest.mark.parametrize("what", ["ffn", "int8_ffn", "backward", "int8", "combine"])
def test_graph_and_streams(what):
    """Captured, replayed with new values and eager work between, and on another stream:
    always the eager result."""
    c = Case(15, N=90, K=2, E=4, A=8, H=144, I=80, int8=what == "int8_ffn")
    gu, dy, wts = c.rows(160), c.rows(144), torch.rand((90, 2), device="cuda")
    dyt = normal(c.g, 90, 144)
    w8 = ep.Int8Weight.from_weight(normal(c.g, 4, 50, 144))

    def call():
        if what == "int8":
            return (ep.int8_linear(c.x, w8, layout=c.layout),)
        if what == "backward":
            return ep.expert_ffn_backward(dy, c.x, gu, c.w13, c.w2, layout=c.layout)
        if what == "combine":
            return ep.combine_backward(dyt, c.x, c.layout, wts)
        return (ep.expert_ffn(c.x, c.w13, c.w2, layout=c.layout),)

    def values(ts):
        return [t[c.at].clone() if t.shape[0] == c.cap else t.clone() for t in ts]
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = call()
    for i in range(4):
        c.x[c.at] = normal(c.g, len(c.at), 144)
        dy[c.at] = normal(c.g, len(c.at), 144)
        eager = values(call())
        graph.replay()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = values(call())
        torch.cuda.current_stream().wait_stream(side)
        for a, b, o in zip(eager, values(captured), other):
            assert torch.equal(a, b) and torch.equal(a, o)
