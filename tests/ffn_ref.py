"""The experts' block, its gradient and 8-bit products in 64 bits, with bounds of the error
that the kernels' roundings allow (the tests' oracle).

Bounds count roundings: half a step of bf16 is 2^-8 of a value; a float32 sum of n terms
is off by at most n 2^-24 of the sum of their magnitudes (products of bf16 are exact in
float32)."""
import torch

BF16 = 2.0 ** -8
F32 = 2.0 ** -24
# the exponential, the quotient and the products of an activation in float32, relative
ACT = 2.0 ** -18


def slots_of(layout, cap):
    """[(expert, its slots)] from a Layout, an LLLayout or None."""
    import combine_ep_get_amd as ep
    if layout is None:
        return [(None, torch.arange(cap))]
    if isinstance(layout, ep.LLLayout):
        E, R, M = layout.num_experts, layout.num_ranks, layout.max_tokens_per_rank
        c = layout.recv_count.cpu().tolist()
        return [(e, torch.cat([torch.arange(c[e][s]) + (e * R + s) * M for s in range(R)]))
                for e in range(E)]
    off, cnt = layout.expert_slot_offset.cpu().tolist(), layout.num_recv_per_expert.cpu().tolist()
    return [(e, torch.arange(cnt[e]) + off[e]) for e in range(layout.num_experts)]


def pick(w, e):
    return (w if e is None else w[e]).double()


def silu_parts(g):
    s = torch.sigmoid(g)
    return s, g * s, s * (1 + g * (1 - s))


def ffn(x, w13, w2):
    """(y, bound of y, gu, bound of gu) for the rows of one expert."""
    H, I = x.shape[1], w2.shape[1]
    gu = x @ w13.t()
    dgu = H * F32 * (x.abs() @ w13.abs().t())
    g, u = gu[:, :I], gu[:, I:]
    _, a, _ = silu_parts(g)
    h = a * u
    # |silu'| <= 1.1
    dh = 1.1 * dgu[:, :I] * (u.abs() + dgu[:, I:]) + a.abs() * dgu[:, I:]
    dh = dh * (1 + BF16) + (BF16 + ACT) * h.abs()
    y = h @ w2.t()
    dy = dh @ w2.abs().t() + I * F32 * ((h.abs() + dh) @ w2.abs().t())
    return y, dy * (1 + BF16) + BF16 * y.abs(), gu, dgu * (1 + BF16) + BF16 * gu.abs()


def ffn_grad(dy, x, gu, w13, w2):
    """((dx, bound), (dw13, bound), (dw2, bound)) for the rows of one expert."""
    n, H, I = x.shape[0], x.shape[1], w2.shape[1]
    g, u = gu[:, :I], gu[:, I:]
    _, a, slope = silu_parts(g)
    dh = dy @ w2
    ddh = H * F32 * (dy.abs() @ w2.abs())
    f = torch.cat([u * slope, a], dim=1)
    # 1 + g (1 - s) cancels where g is about -1.28: its error counts against 1 + |g|
    f_err = ACT * torch.cat([u.abs() * (1 + g.abs()) * torch.sigmoid(g), a.abs()], dim=1)
    dh2, ddh2 = dh.repeat(1, 2), ddh.repeat(1, 2)
    dgu = dh2 * f
    d = (ddh2 * (f.abs() + f_err) + dh2.abs() * f_err) * (1 + BF16) + BF16 * dgu.abs()

    def product(p, dp, q, dq, terms):
        r = p @ q
        err = dp @ q.abs() + (p.abs() + dp) @ dq + terms * F32 * ((p.abs() + dp) @ (q.abs() + dq))
        return r, err * (1 + BF16) + BF16 * r.abs()
    none = torch.zeros_like
    h = a * u
    return (product(dgu, d, w13, none(w13), 2 * I),
            product(dgu.t(), d.t(), x, none(x), n),
            product(dy.t(), none(dy.t()), h, (BF16 + ACT) * h.abs(), n))


def quantize(x):
    """(codes, scales) of rows in 64 bits, as the definition has them."""
    amax = x.double().abs().amax(dim=1) if x.shape[1] else x.new_zeros(x.shape[0]).double()
    scale = (amax / 127).float()
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    q = (x.double() / scale.double()[:, None]).round().clamp(-127, 127)
    return q, scale


def check(got, want, bound, what):
    err = (got.double() - want).abs()
    bad = ~(err <= bound + 1e-30)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err - bound).max()):.3e} "
        f"over its bound at {bad.nonzero()[0].tolist()}")
