"""The experts' block, its gradients and the 8-bit products at a model's width and on buffers
of more than 2^31 bytes, with rows at their far ends."""
from types import SimpleNamespace

import pytest
import torch

import combine_ep_get_amd as ep
from tests import ffn_ref as ref
from tests import ffn_tight as tight
from tests.test_gpu_ffn import BF, NAN, Case, check_ffn, gen, ident, normal

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ a model's width
WIDE = [
    dict(N=1, K=1, E=0, A=1, H=7168, I=2048),
    dict(N=33, K=2, E=4, A=1, H=7168, I=2048),                    # about 16 rows an expert
    dict(N=400, K=2, E=3, A=16, H=7168, I=2048, skew=0.7),
    dict(N=1000, K=1, E=0, A=1, H=7168, I=2048),
]


@pytest.mark.parametrize("shape", WIDE, ids=ident)
def test_width_forward_and_backward(shape):
    c = Case(101, **shape)
    y, gu = c.full(c.H), c.full(2 * c.I)
    ep.expert_ffn(c.x, c.w13, c.w2, layout=c.layout, out=y, gate_up=gu)
    check_ffn(c, y, gu)
    dy, dx = c.rows(c.H), c.full(c.H)
    dw13, dw2 = torch.full_like(c.w13, NAN), torch.full_like(c.w2, NAN)
    ep.expert_ffn_backward(dy, c.x, gu, c.w13, c.w2, layout=c.layout, out=(dx, dw13, dw2))
    for t in (y, gu, dx):
        c.untouched(t)
    for e, s in c.where:
        g13, g2 = (dw13, dw2) if e is None else (dw13[e], dw2[e])
        want = ref.ffn_grad(dy[s].double(), c.x[s].double(), gu[s].double(), ref.pick(c.w13, e),
                            ref.pick(c.w2, e))
        for got, (v, b), what in zip((dx[s], g13, g2), want, ("dx", "dw13", "dw2")):
            ref.check(got, v, b, f"{what} of expert {e}")


@pytest.mark.parametrize("shape", WIDE, ids=ident)
def test_width_int8(shape):
    c = Case(102, int8=True, **shape)
    y, gu = c.full(c.H), c.full(2 * c.I)
    ep.expert_ffn(c.x, c.w13, c.w2, layout=c.layout, out=y, gate_up=gu)
    c.untouched(y)
    c.untouched(gu)
    for e, s in c.where:
        w = [(w.codes, w.scales) if e is None else (w.codes[e], w.scales[e]) for w in (c.w13, c.w2)]
        want, choices = tight.block(c.x[s], *w)
        tight.check_gate_up(gu[s], want, f"gate_up of expert {e}")
        tight.check_rows(y[s], choices, f"y of expert {e}")


# ------------------------------------------------------------------ far ends
def far(cap, counts, bound):
    """Regions that end where the buffer does, one after the other."""
    i32 = dict(dtype=torch.int32, device="cuda")
    off = [cap - sum(counts[e:]) for e in range(len(counts))]
    lay = SimpleNamespace(num_experts=len(counts), num_tokens=bound, num_topk=1, capacity=cap,
                          expert_slot_offset=torch.tensor([*off, cap], **i32),
                          num_recv_per_expert=torch.tensor(counts, **i32))
    return lay, [torch.arange(o, o + n, device="cuda") for o, n in zip(off, counts)]


def empty(rows, cols, at, g):
    t = torch.empty((rows, cols), dtype=BF, device="cuda")
    assert t.numel() * 2 > 2 ** 31
    t[at] = normal(g, len(at), cols)
    return t


# few rows and the 64-row tiles by what the call says it has; 256-row tiles
@pytest.mark.parametrize("bound,counts", [(60, [5, 40, 15]), (700, [300, 0, 400]),
                                          (100000, [300, 257, 400])])
def test_regions_far_out(bound, counts):
    H, I, cap, g = 264, 136, 8_200_000, gen(103)
    lay, where = far(cap, counts, bound)
    at = torch.cat(where)
    x, dy, gu = empty(cap, H, at, g), empty(cap, H, at, g), empty(cap, 2 * I, at, g)
    w13, w2 = normal(g, 3, 2 * I, H, scale=H ** -0.5), normal(g, 3, H, I, scale=I ** -0.5)
    y, out = torch.empty_like(x), torch.empty_like(gu)
    last = at[0] - 1
    y[:last + 1], out[:last + 1] = 7.0, 7.0
    ep.expert_ffn(x, w13, w2, layout=lay, out=y, gate_up=out)
    assert bool((y[:last + 1] == 7.0).all()) and bool((out[:last + 1] == 7.0).all())
    for e, s in enumerate(where):
        want, by, wgu, bgu = ref.ffn(x[s].double(), w13[e].double(), w2[e].double())
        ref.check(y[s], want, by, f"y of expert {e}")
        ref.check(out[s], wgu, bgu, f"gate_up of expert {e}")
    dx, dw13, dw2 = ep.expert_ffn_backward(dy, x, gu, w13, w2, layout=lay,
                                           out=(y, torch.empty_like(w13), torch.empty_like(w2)))
    assert bool((dx[:last + 1] == 7.0).all())
    for e, s in enumerate(where):
        want = ref.ffn_grad(dy[s].double(), x[s].double(), gu[s].double(), w13[e].double(),
                            w2[e].double())
        for got, (v, b), what in zip((dx[s], dw13[e], dw2[e]), want, ("dx", "dw13", "dw2")):
            ref.check(got, v, b, f"{what} of expert {e}")
    q = ep.Int8Weight.from_weight(normal(g, 3, 131, H // 16 * 16))
    x8 = x.view(-1)[:cap * 256].view(cap, 256)             # other rows of the same memory
    x8[at] = normal(g, len(at), 256)
    z = ep.int8_linear(x8, q, layout=lay)
    for e, s in enumerate(where):
        codes, scale = ref.quantize(x8[s])
        want = (codes @ q.codes[e].double().t()) * scale.double()[:, None] * q.scales[e].double()
        ref.check(z[s], want, tight.ONCE * want.abs(), f"y of expert {e}")


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("bound", [60, 100000])
def test_sub_blocks_far_out(int8, bound):
    """Sub-blocks of 0.5 GiB, 1 GiB an expert: the second source's rows, the last expert's."""
    E, R, M, H, I, g = 3, 2, 1 << 20, 256, 144, gen(104)
    counts = torch.tensor([[0, 30], [270, 300], [3, 290]], dtype=torch.int32, device="cuda")
    lay = ep.LLLayout(bound, 1, E, R, M, E * R * M, counts, None, None)
    where = [torch.cat([torch.arange(n, device="cuda") + (e * R + s) * M for s, n in enumerate(of)])
             for e, of in enumerate(counts.tolist())]
    x = empty(E * R * M, H, torch.cat(where), g)
    w = normal(g, E, 2 * I, H, scale=H ** -0.5), normal(g, E, H, I, scale=I ** -0.5)
    if int8:
        w = tuple(ep.Int8Weight.from_weight(t) for t in w)
    gu = torch.empty((E * R * M, 2 * I), dtype=BF, device="cuda")
    y = ep.expert_ffn(x, *w, layout=lay, gate_up=gu)
    for e, s in enumerate(where):
        if int8:
            want, choices = tight.block(x[s], *[(t.codes[e], t.scales[e]) for t in w])
            tight.check_gate_up(gu[s], want, f"gate_up of expert {e}")
            tight.check_rows(y[s], choices, f"y of expert {e}")
        else:
            want, by, wgu, bgu = ref.ffn(x[s].double(), w[0][e].double(), w[1][e].double())
            ref.check(y[s], want, by, f"y of expert {e}")
            ref.check(gu[s], wgu, bgu, f"gate_up of expert {e}")


def test_plain_far_out():
    """A plain matrix of more than 2^31 bytes: its last rows, in bf16 and in codes."""
    N, C, O, g = 9_000_003, 256, 136, gen(105)
    tail = slice(N - 300, N)
    x = torch.zeros((N, C), dtype=BF, device="cuda")
    x[tail] = normal(g, 300, C)
    w = ep.Int8Weight.from_weight(normal(g, O, C))
    codes, scales = ep.quantize_int8(x)
    q, s = ref.quantize(x[tail])
    assert torch.equal(codes[tail].double(), q) and torch.equal(scales[tail], s)
    assert not bool(codes[:N - 300].any()) and bool((scales[:N - 300] == 1).all())
    want = (q @ w.codes.double().t()) * s.double()[:, None] * w.scales.double()
    for y in (ep.int8_linear(x, w), ep.int8_linear(codes, w, x_scales=scales)):
        ref.check(y[tail], want, tight.ONCE * want.abs(), "y")
        assert not bool(y[:N - 300].any())
    w13, w2 = normal(g, 2 * 24, C, scale=C ** -0.5), normal(g, C, 24, scale=24 ** -0.5)
    y = ep.expert_ffn(x, w13, w2)
    want, bound, _, _ = ref.ffn(x[tail].double(), w13.double(), w2.double())
    ref.check(y[tail], want, bound, "y")
    assert not bool(y[:N - 300].any())


def test_combine_backward_far_out():
    """Slots behind 2^31 bytes of expert_out."""
    N, K, H, cap, g = 500, 3, 7168, 200_000, gen(106)
    slot = (cap - 1 - torch.randperm(N * K, generator=g, device="cuda")).int().view(N, K)
    lay = ep.LLLayout(N, K, 4, 1, cap, cap, None, slot, None)
    dy, wts = normal(g, N, H), torch.rand((N, K), generator=g, device="cuda")
    eo = empty(cap, H, slot.view(-1).long(), g)
    deo = torch.empty_like(eo)
    deo[:cap - N * K] = 7.0
    dw = ep.combine_backward(dy, eo, lay, wts, out=(deo, torch.empty_like(wts)))[1]
    assert bool((deo[:cap - N * K] == 7.0).all())
    at = slot.long()
    want = wts.double()[:, :, None] * dy.double()[:, None]
    ref.check(deo[at], want, (ref.BF16 + 2 * ref.F32) * want.abs(), "d_expert_out")
    o = eo[at].double() * dy.double()[:, None]
    ref.check(dw, o.sum(dim=2), H * ref.F32 * o.abs().sum(dim=2), "d_topk_weights")
