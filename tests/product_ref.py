"""Plain 64-bit implementations of the router and of the experts' products, for
the tests, with the error bounds that the kernels' arithmetic allows.

Bounds.  A product of two bf16 values is exact in float32; a float32 sum of n
terms is off by at most (n - 1) U times the sum of the magnitudes, whatever its
order, with U = 2^-23 (one step per addition: the matrix instruction need not
round to nearest).  A rounding to bf16 is off by at most 2^-8 of the value
(half of torch.finfo(bfloat16).eps).
"""
import copy
import math

import torch

import combine_ep_get_amd as ep

U = 2.0 ** -23
HALF = torch.finfo(torch.bfloat16).eps / 2
TINY = 2.0 ** -120            # results below it may be flushed or lose bits
E2M1 = torch.tensor([0., .5, 1., 1.5, 2., 3., 4., 6., -0., -.5, -1., -1.5, -2., -3., -4., -6.],
                    dtype=torch.float64)


class W:
    """A random weight [*lead, rows, cols] on the GPU (`arg`: what the library
    takes), its 64-bit value (`value`) and the magnitudes that its kernel sums
    (`mags`: for int4 the 128 + code and 128 + zero parts separately)."""

    def __init__(self, fmt, lead, rows, cols, group=None, zeros=False, gen=None, device="cuda"):
        shape = (*lead, rows, cols)
        self.fmt, self.cols = fmt, cols
        if fmt == "bf16":
            w = (torch.randn(shape, generator=gen) * cols ** -0.5).to(torch.bfloat16)
            self.arg, self.value = w.to(device), w.double()
            self.mags = self.value.abs()
            self.parts = 1
            return
        group = group or (128 if fmt == "int4" else 32)
        self.group = group
        codes = torch.randint(0, 16, shape, generator=gen, dtype=torch.uint8)
        per = (*lead, rows, cols // group)
        self.parts = cols // group
        if fmt == "int4":
            s = ((torch.rand(per, generator=gen) + 0.5) * cols ** -0.5 / 4).to(torch.bfloat16)
            z = torch.randint(0, 16, per, generator=gen, dtype=torch.uint8) if zeros else None
            z64 = torch.full(per, 8.0, dtype=torch.float64) if z is None else z.double()
            wide = lambda t: t.double().repeat_interleave(group, dim=-1)   # noqa: E731
            self.value = (codes.double() - wide(z64)) * wide(s)
            self.mags = (256.0 + codes.double() + wide(z64)) * wide(s)
        else:
            s = (torch.randint(-2, 2, per, generator=gen)
                 + 126 - round(0.5 * math.log2(cols))).to(torch.uint8)
            z = None
            self.value = E2M1[codes.long()] * torch.pow(
                2.0, s.double() - 127).repeat_interleave(group, dim=-1)
            self.mags = self.value.abs()
            self.parts = 1
        packed = ep.pack_codes(codes, fmt)
        self.arg = ep.QuantWeight(packed.to(device), s.to(device),
                                  zeros=None if z is None else z.to(device), group=group, fmt=fmt)

    def only(self, e, device):
        """The values of one of a stack, on `device` (no `arg`)."""
        w = copy.copy(self)
        w.value, w.mags, w.arg = self.value[e].to(device), self.mags[e].to(device), None
        return w

    def product(self, x, at=()):
        """(x W^T, bound of the kernel's float32 error) in 64 bits."""
        v, m = self.value[at], self.mags[at]
        y = x @ v.t()
        if self.parts == 1:
            return y, (self.cols + 16) * U * (x.abs() @ m.t())
        # int4: sums inside each group of the 128-offset codes, then over groups
        err = (self.group + 8) * U * (x.abs() @ m.t())
        over = (self.parts + 16) * U * (x.abs() @ v.abs().t())
        return y, err + over


def moe(x, idx, wts, w13, w2):
    """(y, bound) of the expert layer in 64 bits; idx [N, K] host, -1 or any id
    outside the experts: no expert."""
    x = x.double()
    N, H = x.shape
    E, _, I = w2.value.shape
    y, bound = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(N):
        named = {}
        for k in range(idx.shape[1]):
            e = int(idx[t, k])
            if 0 <= e < E:
                named[e] = named.get(e, 0.0) + float(wts[t, k])
        for e, w in named.items():
            gu, err = w13.product(x[t:t + 1], e)
            g, u, eg, eu = gu[:, :I], gu[:, I:], err[:, :I], err[:, I:]
            sg = g * torch.sigmoid(g)
            h = w * sg * u
            # |silu'| <= 1.1; silu itself within 8 steps of float32
            eh = abs(w) * (1.1 * u.abs() * eg + sg.abs() * eu + 1.1 * eg * eu
                           + 16 * U * (sg * u).abs())
            eh = eh + HALF * (h.abs() + eh)          # the rounding between the products
            p, ep_ = w2.product(h, e)
            y[t] += p[0]
            bound[t] += (ep_ + eh @ w2.value[e].abs().t())[0] * (1 + 2.0 ** -6)
        bound[t] += 64 * U * y[t].abs()              # the sum over experts and wavefronts
    return y, bound + HALF * (y.abs() + bound) + TINY


def moe_by_expert(x, idx, wts, w13, w2, device="cpu"):
    """moe() with an expert's tokens together, on `device`: for larger sizes."""
    x, wts = x.double().to(device), wts.double().to(device)
    E, H, I = w2.value.shape
    y, bound = torch.zeros_like(x), torch.zeros_like(x)
    for e in range(E):
        w = (wts * (idx == e).to(device)).sum(dim=1)
        at = (idx == e).any(dim=1).nonzero()[:, 0].to(device)
        if not len(at):
            continue
        w = w[at, None]
        a, b = w13.only(e, device), w2.only(e, device)
        gu, err = a.product(x[at])
        g, u, eg, eu = gu[:, :I], gu[:, I:], err[:, :I], err[:, I:]
        sg = g * torch.sigmoid(g)
        h = w * sg * u
        eh = w.abs() * (1.1 * u.abs() * eg + sg.abs() * eu + 1.1 * eg * eu
                        + 16 * U * (sg * u).abs())
        eh = eh + HALF * (h.abs() + eh)
        p, ep_ = b.product(h)
        y[at] += p
        bound[at] += (ep_ + eh @ b.value.abs().t()) * (1 + 2.0 ** -6)
    bound += 64 * U * y.abs()
    return y.cpu(), (bound + HALF * (y.abs() + bound) + TINY).cpu()


def linear(x, w):
    y, err = w.product(x.double())
    return y, err + HALF * (y.abs() + err) + TINY


def route(logits, K, bias=None, scoring="sigmoid", num_groups=1, topk_groups=1, group_top=1,
          renormalize=True, scale=1.0):
    """The router one token at a time, in Python floats."""
    ids, weights = [], []
    for row in logits.double().tolist():
        E, G = len(row), num_groups
        l = [min(v, 3.402823466e38) for v in row]
        live = [v > -math.inf for v in l]             # False for NaN
        if scoring == "softmax":
            top = max([v for v, a in zip(l, live) if a], default=0.0)
            ex = [math.exp(v - top) if a else 0.0 for v, a in zip(l, live)]
            total = math.fsum(ex)
            s = [v / total if total else 0.0 for v in ex]
        else:
            s = [(1 / (1 + math.exp(-v)) if v > -700 else 0.0) if a else 0.0
                 for v, a in zip(l, live)]
        v = [(a + float(b)) for a, b in zip(s, bias.tolist())] if bias is not None else s
        order = v if bias is not None else l
        per = E // G
        scores = []
        for g in range(G):
            best = sorted((v[e] if group_top == 2 or bias is not None else l[e]
                           for e in range(g * per, (g + 1) * per) if live[e]), reverse=True)
            scores.append(sum(best[:group_top]) if len(best) >= group_top else -math.inf)
        kept = sorted(range(G), key=lambda g: (-scores[g], g))[:topk_groups]
        can = [e for e in range(E) if live[e] and e // per in kept]
        best = sorted(can, key=lambda e: (-order[e], e))[:K]
        w = [s[e] for e in best]
        if renormalize and best:
            # quotients of scores from their logarithms: the scores themselves may underflow
            if scoring == "softmax":
                logs = [l[e] for e in best]
            else:
                logs = [min(l[e], 0.0) - math.log1p(math.exp(-abs(l[e]))) for e in best]
            ratio = [math.exp(a - max(logs)) for a in logs]
            w = [a / math.fsum(ratio) for a in ratio]
        ids.append(best + [-1] * (K - len(best)))
        weights.append([a * scale for a in w] + [0.0] * (K - len(best)))
    return torch.tensor(ids, dtype=torch.int64).view(-1, K), \
        torch.tensor(weights, dtype=torch.float64).view(-1, K)
