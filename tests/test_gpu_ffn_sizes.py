"""The experts' block, its gradient and the 8-bit products where they run on 256-row tiles
(many rows), whole and ragged, and calls that a user makes around them."""
import pytest
import torch

import combine_ep_get_amd as ep
from tests import ffn_ref as ref
from tests.test_gpu_ffn import BF, Case, check_ffn, check_int8_ffn, gen, ident, normal, routing

pytestmark = pytest.mark.gpu

MANY = [
    dict(N=4096, K=1, E=0, A=1, H=1024, I=512),                       # whole tiles only
    dict(N=5000, K=1, E=0, A=1, H=1000, I=520),                       # ragged in every way
    dict(N=4100, K=1, E=0, A=1, H=72, I=2056),                        # two steps; long down
    dict(N=2500, K=3, E=4, A=16, H=1000, I=520, skew=1.0),            # uneven experts
    dict(N=3000, K=2, E=40, A=1, H=1064, I=264, skew=0.7),            # tall and short tiles
]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("H,I", [(272, 144), (128, 64)])     # several steps; the fewest
def test_tall_tiles_then_short_ones(int8, H, I, monkeypatch):
    """Row counts around a tile's ends, so many that a workgroup takes both kinds."""
    counts = torch.tensor([0, 1, 64, 65, 127, 128, 129, 192, 255, 256, 257, 384, 385] * 25)
    idx = torch.repeat_interleave(torch.arange(len(counts)), counts)
    idx = idx[torch.randperm(len(idx), generator=torch.Generator().manual_seed(31))]
    idx = idx.to(torch.int32).view(-1, 1).cuda()
    monkeypatch.setattr("tests.test_gpu_ffn.routing", lambda *a: idx)
    c = Case(31, N=len(idx), K=1, E=len(counts), A=1, H=H, I=I, int8=int8)
    assert [len(s) for _, s in c.where] == counts.tolist()
    y = ep.expert_ffn(c.x, c.w13, c.w2, layout=c.layout, out=c.full(H))
    c.untouched(y)
    c.where = c.where[:26] + c.where[-13:]
    (check_int8_ffn if int8 else check_ffn)(c, y)
    for _ in range(3):
        again = ep.expert_ffn(c.x, c.w13, c.w2, layout=c.layout)
        assert torch.equal(again[c.at], y[c.at])


# on 64-row tiles
MIDDLE = [
    dict(N=512, K=1, E=0, A=1, H=2048, I=1024),
    dict(N=333, K=1, E=0, A=1, H=2008, I=1032),
    dict(N=300, K=3, E=6, A=8, H=1544, I=776, skew=0.7),
]


@pytest.mark.parametrize("shape", MANY + MIDDLE, ids=ident)
def test_forward(shape):
    c = Case(21, **shape)
    y, gu = c.full(c.H), c.full(2 * c.I)
    ep.expert_ffn(c.x, c.w13, c.w2, layout=c.layout, out=y, gate_up=gu)
    check_ffn(c, y, gu)
    c.untouched(y)
    c.untouched(gu)
    for _ in range(3):
        again = ep.expert_ffn(c.x, c.w13, c.w2, layout=c.layout)
        assert torch.equal(again[c.at], y[c.at])


@pytest.mark.parametrize("shape", MANY, ids=ident)
def test_backward(shape):
    c = Case(22, **shape)
    gu, dy = c.rows(2 * c.I), c.rows(c.H)
    dx = c.full(c.H)
    out = dx, torch.full_like(c.w13, float("nan")), torch.full_like(c.w2, float("nan"))
    ep.expert_ffn_backward(dy, c.x, gu, c.w13, c.w2, layout=c.layout, out=out)
    c.untouched(dx)
    for e, s in c.where:
        g13, g2 = out[1:] if e is None else (out[1][e], out[2][e])
        if len(s) == 0:
            assert not bool(g13.any()) and not bool(g2.any())
            continue
        want = ref.ffn_grad(dy[s].double(), c.x[s].double(), gu[s].double(), ref.pick(c.w13, e),
                            ref.pick(c.w2, e))
        for got, (w, b), what in zip((dx[s], g13, g2), want, ("dx", "dw13", "dw2")):
            ref.check(got, w, b, f"{what} of expert {e}")
    for _ in range(3):
        again = ep.expert_ffn_backward(dy, c.x, gu, c.w13, c.w2, layout=c.layout)
        assert torch.equal(again[0][c.at], dx[c.at])
        assert all(torch.equal(a, b) for a, b in zip(again[1:], out[1:]))


@pytest.mark.parametrize("shape", [
    dict(N=4096, K=1, E=0, A=1, H=1024, I=512),
    dict(N=6000, K=1, E=0, A=1, H=1008, I=528),
    dict(N=3000, K=3, E=4, A=16, H=1008, I=528, skew=1.0),
    dict(N=512, K=1, E=0, A=1, H=4096, I=2048),                       # 64-row tiles
    dict(N=333, K=1, E=0, A=1, H=4080, I=2064),
    dict(N=300, K=3, E=6, A=8, H=3088, I=1552, skew=0.7),
], ids=ident)
def test_int8_ffn(shape):
    c = Case(23, int8=True, **shape)
    y = ep.expert_ffn(c.x, c.w13, c.w2, layout=c.layout, out=c.full(c.H))
    check_int8_ffn(c, y)
    c.untouched(y)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("shape", [dict(N=4000, K=2, E=8, R=8, ll=500, H=1008, I=528),
                                   dict(N=400, K=2, E=4, R=4, ll=100, H=2064, I=1040)], ids=ident)
def test_low_latency_many_rows(int8, shape):
    """Row tiles that cross the sources' sub-blocks."""
    c = Case(24, A=1, drop=0.2, int8=int8, **shape)
    y = ep.expert_ffn(c.x, c.w13, c.w2, layout=c.layout, out=c.full(c.H))
    c.untouched(y)
    (check_int8_ffn if int8 else check_ffn)(c, y)


@pytest.mark.parametrize("N,C,O", [(4096, 512, 1024), (4111, 1040, 1237), (5000, 16, 3001),
                                   (980, 7120, 861), (700, 4096, 1022)])
def test_int8_linear(N, C, O):
    g = gen(25)
    codes = torch.randint(-128, 128, (O, C), generator=g, device="cuda").to(torch.int8)
    w = ep.Int8Weight(codes, torch.rand((O,), generator=g, device="cuda") + 0.1)
    x = normal(g, N, C)
    y = ep.int8_linear(x, w)
    q, s = ref.quantize(x)
    want = (q @ codes.double().t()) * s.double()[:, None] * w.scales.double()
    ref.check(y, want, (ref.BF16 + 4 * ref.F32) * want.abs(), "y")


@pytest.mark.parametrize("N", [1, 2, 7, 16, 17])
def test_rounded_on_the_way_or_before(N):
    """int8_linear of bf16 rows is that of their codes, whichever kernel rounds them."""
    g = gen(26)
    w = ep.Int8Weight.from_weight(normal(g, 333, 1008))
    x = normal(g, N, 1008)
    x[0] = (x[0].float() * 1e-38).to(BF)
    codes, scales = ep.quantize_int8(x)
    assert torch.equal(ep.int8_linear(x, w), ep.int8_linear(codes, w, x_scales=scales))


def test_in_place_and_at_once():
    """y over x; two calls at once on two streams with their own workspaces."""
    a, b = (Case(27 + i, N=900, K=2, E=6, A=8, H=256, I=144) for i in range(2))
    want = [ep.expert_ffn(c.x, c.w13, c.w2, layout=c.layout)[c.at].clone() for c in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for c, st in zip((a, b), streams):
        with torch.cuda.stream(st):
            out = ep.expert_ffn(c.x, c.w13, c.w2, layout=c.layout, out=c.x)
            assert out is c.x
    torch.cuda.synchronize()
    for c, w in zip((a, b), want):
        assert torch.equal(c.x[c.at], w)


def test_larger_buffers_and_workspaces():
    """Buffers with more rows than the layout needs, a workspace for more, a wrong one."""
    g = gen(29)
    idx = routing(g, 200, 2, 5)
    lay = ep.get_layout(idx, 5, 1, 4)
    cap = lay.capacity + 77
    x = torch.full((cap, 64), float("nan"), dtype=BF, device="cuda")
    at = torch.cat([s for _, s in ref.slots_of(lay, cap)]).cuda()
    x[at] = normal(g, len(at), 64)
    w13, w2 = normal(g, 5, 96, 64), normal(g, 5, 64, 48)
    y = torch.full_like(x, 7.0)
    ws = ep.alloc_ffn_workspace(2 * cap, 64, 48)
    ep.expert_ffn(x, w13, w2, layout=lay, out=y, workspace=ws)
    small = ep.expert_ffn(x[:lay.capacity].contiguous(), w13, w2, layout=lay)
    assert torch.equal(y[at], small[at])
    rest = torch.ones(cap, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert bool((y[rest] == 7.0).all())
    with pytest.raises(ValueError):
        ep.expert_ffn(x[:lay.capacity - 1].contiguous(), w13, w2, layout=lay)
    with pytest.raises(ValueError):
        ep.expert_ffn(x, w13, w2, layout=lay, workspace=ws[:1000])
    with pytest.raises(ValueError):
        ep.expert_ffn(x, w13.float(), w2, layout=lay)
    with pytest.raises(ValueError):
        ep.expert_ffn(x[:, ::2], w13, w2, layout=lay)
    with pytest.raises(ValueError):                      # rows of 60: no whole 16 bytes
        ep.expert_ffn(x[:, :60].contiguous(), w13[:, :, :60].contiguous(),
                      w2[:, :60].contiguous(), layout=lay)


def test_most_experts_on_wide_tiles():
    """1024 experts with about 128 rows each, none in some."""
    g = gen(30)
    E, N, H, I = 1024, 131072, 256, 64
    idx = torch.randint(0, E, (N, 1), generator=g, device="cuda").to(torch.int32)
    idx[idx % 101 == 7] = -1
    lay = ep.get_layout(idx, E, 1, 1)
    where = ref.slots_of(lay, lay.capacity)
    at = torch.cat([s for _, s in where]).cuda()
    x, dy, gu = (torch.zeros((lay.capacity, n), dtype=BF, device="cuda") for n in (H, H, 2 * I))
    for t in (x, dy, gu):
        t[at] = normal(g, len(at), t.shape[1])
    w13, w2 = normal(g, E, 2 * I, H, scale=H ** -0.5), normal(g, E, H, I, scale=I ** -0.5)
    y = ep.expert_ffn(x, w13, w2, layout=lay)
    dx, dw13, dw2 = ep.expert_ffn_backward(dy, x, gu, w13, w2, layout=lay)
    for e, s in where[::53] + where[7::101] + where[-1:]:
        s = s.cuda()
        if len(s) == 0:
            assert not bool(dw13[e].any()) and not bool(dw2[e].any())
            continue
        a = [t.double() for t in (x[s], w13[e], w2[e])]
        want, bound, _, _ = ref.ffn(*a)
        ref.check(y[s], want, bound, f"y of expert {e}")
        want = ref.ffn_grad(dy[s].double(), a[0], gu[s].double(), a[1], a[2])
        for got, (v, b), what in zip((dx[s], dw13[e], dw2[e]), want, ("dx", "dw13", "dw2")):
            ref.check(got, v, b, f"{what} of expert {e}")
