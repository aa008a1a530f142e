"""The experts' block with 8-bit weights, value by value (the tests' oracle): which codes of h
may differ, and the bound of y that follows.

A code of h depends on h after its rounding to bf16.  What float32 makes of h is off by at
most `e`; where bf16(h - e) and bf16(h + e) lead to the same integer the code is known, and
only the others (next to a midpoint of bf16 and to a half at once) are allowed a step.  A
row's scale comes from its largest bf16(h); where that may be either of two neighbours, the
row has to fit one of them."""
import torch

from tests.ffn_ref import ACT, BF16, F32, quantize

ONCE = BF16 + 4 * F32        # one rounding to bf16; the sum's, both scales' products in float32


def products(x, q, s):
    """x's codes by a weight's, times both scales: exact but for 64 bits."""
    qx, sx = quantize(x)
    return (qx @ q.double().t()) * sx.double()[:, None] * s.double()


def block(x, w13, w2):
    """(gate_up, [(y, bound) for each scale that h's rows may have]) for one expert's rows;
    w13, w2: (codes, scales)."""
    gu = products(x, *w13)
    I = gu.shape[1] // 2
    g, u = gu[:, :I], gu[:, I:]
    h = g * torch.sigmoid(g) * u
    # g and u are off by 3 roundings each (times 1 + |g| through silu), the exponent of the
    # exponential by one of g, the rest is ACT's
    e = h.abs() * (ACT + 4 * F32 * (2 + g.abs()))
    lo, hi = ((h + d).to(torch.bfloat16).double() for d in (-e, e))
    q2, s2 = w2[0].double(), w2[1].double()

    def result(top):
        scale = (top / 127).float().double()[:, None]
        scale = torch.where(scale == 0, torch.ones_like(scale), scale)
        a, b = ((t / scale).round().clamp(-127, 127) for t in (lo, hi))
        y, slack = (a @ q2.t()) * scale * s2, ((b - a).abs() @ q2.abs().t()) * scale * s2.abs()
        return y, slack + ONCE * (y.abs() + slack)
    least = torch.minimum(lo.abs(), hi.abs()).amax(dim=1)
    most = torch.maximum(lo.abs(), hi.abs()).amax(dim=1)
    return gu, [result(top) for top in (least, most)]


def check_gate_up(got, want, what):
    bad = ~((got.double() - want).abs() <= ONCE * want.abs() + 1e-30)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} off, first at {bad.nonzero()[0].tolist()}"


def check_rows(got, choices, what):
    """Every row of y within its bound for one of the choices."""
    bads = [~((got.double() - y).abs() <= bound + 1e-30) for y, bound in choices]
    bad = torch.where(bads[0].sum(dim=1, keepdim=True) <= bads[1].sum(dim=1, keepdim=True), *bads)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} off in "
                                 f"{int(bad.any(dim=1).sum())} rows, first at {bad.nonzero()[0].tolist()}")
