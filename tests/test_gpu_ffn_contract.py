"""Calls that the contract of the experts' block and the 8-bit products allows and that an
ordinary program rarely makes: counts and offsets that leave the buffer, more rows than the
bound."""
from types import SimpleNamespace

import pytest
import torch

import combine_ep_get_amd as ep
from tests import ffn_ref as ref
from tests.test_gpu_ffn import BF, NAN, gen, normal

pytestmark = pytest.mark.gpu
TOP = 2 ** 31 - 1


def regions(offset, count, cap, bound):
    """A layout of hand-made regions (bound: rows it claims to have at most) and the slots
    of each expert, as the contract cuts them off."""
    i32 = dict(dtype=torch.int32, device="cuda")
    lay = SimpleNamespace(num_experts=len(count), num_tokens=bound, num_topk=1, capacity=cap,
                          expert_slot_offset=torch.tensor([*offset, 0], **i32),
                          num_recv_per_expert=torch.tensor(count, **i32))
    where = [torch.arange(max(0, min(o, cap)), max(0, min(o, cap), min(o + c, cap)), device="cuda")
             for o, c in zip(offset, count)]
    return lay, where


# offsets, counts, rows of the buffer; the regions stay apart whatever is cut off
OUTSIDE = {
    "before": ([-3, 6], [5, 7], 50),
    "behind": ([40, 8], [30, 5], 50),
    "around": ([-9, 800], [709, TOP], 1100),
    "nowhere": ([10, -20, 60, 4], [-7, 12, 9, 3], 50),
    "extreme": ([-TOP - 1, 5, TOP, 20, 7], [TOP, TOP * -1, TOP, 13, 0], 300),
}


class Buffers:
    def __init__(self, name, bound, H, I, seed=51):
        offset, count, cap = OUTSIDE[name]
        self.lay, self.where = regions(offset, count, cap, bound)
        self.cap, self.H, self.I, self.g = cap, H, I, gen(seed)
        self.at = torch.cat(self.where)
        self.rest = torch.ones((cap,), dtype=torch.bool, device="cuda")
        self.rest[self.at] = False

    def rows(self, cols):
        t = torch.full((self.cap, cols), NAN, dtype=BF, device="cuda")
        t[self.at] = normal(self.g, len(self.at), cols)
        return t

    def full(self, cols):
        return torch.full((self.cap, cols), 7.0, dtype=BF, device="cuda")

    def untouched(self, t):
        assert bool((t[self.rest] == 7.0).all()), "a slot of no expert was written"

    def weights(self, *shape):
        return normal(self.g, len(self.where), *shape, scale=shape[-1] ** -0.5)


# how many rows the call claims to have: fewer than it has too
BOUNDS = [1, 700, 100000]


@pytest.mark.parametrize("bound", BOUNDS)
@pytest.mark.parametrize("name", OUTSIDE)
def test_regions_forward_and_backward(name, bound):
    c = Buffers(name, bound, 136, 72)
    x, dy, w13, w2 = c.rows(c.H), c.rows(c.H), c.weights(2 * c.I, c.H), c.weights(c.H, c.I)
    y, gu, dx = c.full(c.H), c.full(2 * c.I), c.full(c.H)
    ep.expert_ffn(x, w13, w2, layout=c.lay, out=y, gate_up=gu)
    dw13, dw2 = torch.full_like(w13, NAN), torch.full_like(w2, NAN)
    given = c.rows(2 * c.I)
    ep.expert_ffn_backward(dy, x, given, w13, w2, layout=c.lay, out=(dx, dw13, dw2))
    for t in (y, gu, dx):
        c.untouched(t)
    for e, s in enumerate(c.where):
        if len(s) == 0:
            assert not bool(dw13[e].any()) and not bool(dw2[e].any())
            continue
        a = [t.double() for t in (x[s], w13[e], w2[e])]
        want, bound_y, wgu, bgu = ref.ffn(*a)
        ref.check(y[s], want, bound_y, f"y of expert {e}")
        ref.check(gu[s], wgu, bgu, f"gate_up of expert {e}")
        want = ref.ffn_grad(dy[s].double(), a[0], given[s].double(), a[1], a[2])
        for got, (v, b), what in zip((dx[s], dw13[e], dw2[e]), want, ("dx", "dw13", "dw2")):
            ref.check(got, v, b, f"{what} of expert {e}")


@pytest.mark.parametrize("bound", BOUNDS)
@pytest.mark.parametrize("name", OUTSIDE)
def test_regions_int8(name, bound):
    c = Buffers(name, bound, 144, 0)
    x, w = c.rows(c.H), ep.Int8Weight.from_weight(c.weights(77, c.H))
    y = torch.full((c.cap, 77), 7.0, dtype=BF, device="cuda")
    ep.int8_linear(x, w, layout=c.lay, out=y)
    c.untouched(y)
    for e, s in enumerate(c.where):
        q, scale = ref.quantize(x[s])
        want = (q @ w.codes[e].double().t()) * scale.double()[:, None] * w.scales[e].double()
        ref.check(y[s], want, (ref.BF16 + 4 * ref.F32) * want.abs(), f"y of expert {e}")


@pytest.mark.parametrize("bound", BOUNDS)
@pytest.mark.parametrize("int8", [False, True])
def test_sub_blocks_forward(int8, bound):
    """Counts below zero and above a sub-block's rows."""
    E, R, M, H, I = 3, 4, 150, 144, 80
    counts = torch.tensor([[-1, 151, 3, TOP], [0, 0, 0, -TOP - 1], [150, 149, 1, 0]],
                          dtype=torch.int32, device="cuda")
    cap, g = E * R * M + 9, gen(52)
    lay = ep.LLLayout(bound, 1, E, R, M, E * R * M, counts, None, None)
    held = counts.clamp(0, M).tolist()
    where = [torch.cat([torch.arange(n, device="cuda") + (e * R + s) * M
                        for s, n in enumerate(of)]) for e, of in enumerate(held)]
    at = torch.cat(where)
    x = torch.full((cap, H), NAN, dtype=BF, device="cuda")
    x[at] = normal(g, len(at), H)
    w = normal(g, E, 2 * I, H, scale=H ** -0.5), normal(g, E, H, I, scale=I ** -0.5)
    y = torch.full((cap, H), 7.0, dtype=BF, device="cuda")
    gu = torch.full((cap, 2 * I), 7.0, dtype=BF, device="cuda")
    if int8:
        w = tuple(ep.Int8Weight.from_weight(t) for t in w)
    ep.expert_ffn(x, *w, layout=lay, out=y, gate_up=gu)
    for e, s in enumerate(where):
        if len(s) == 0:
            continue
        if int8:
            q, scale = ref.quantize(x[s])
            want = (q @ w[0].codes[e].double().t()) * scale.double()[:, None] \
                * w[0].scales[e].double()
            ref.check(gu[s], want, (ref.BF16 + 4 * ref.F32) * want.abs(), f"gate_up of {e}")
        else:
            want, by, wgu, bgu = ref.ffn(x[s].double(), w[0][e].double(), w[1][e].double())
            ref.check(y[s], want, by, f"y of expert {e}")
            ref.check(gu[s], wgu, bgu, f"gate_up of expert {e}")
    rest = torch.ones((cap,), dtype=torch.bool, device="cuda")
    rest[at] = False
    assert bool((y[rest] == 7.0).all()) and bool((gu[rest] == 7.0).all())
