"""The experts' feed-forward block on dispatched rows, its gradient, combine's
gradient and 8-bit integer products, at the sizes they are used at.

Dispatch leaves the rows of expert e in slots [off[e], off[e] + count[e]) of a
receive buffer whose other slots hold nothing; the operators here work on those
rows (or, with experts == 0, on all rows of a plain matrix):

  ffn          y = (silu(x Wg^T) * (x Wu^T)) W2^T per expert; bf16 weights, or
               8-bit integer weights with rows quantised on the way
  ffn_grad     the gradients of x, W13 = [Wg; Wu] and W2 from that of y and the
               pre-activations
  combine_grad the gradients of the expert outputs and of the gate weights of
               y[t] = sum_k weight[t, k] * expert_out[slot[t, k]]
  int8         y = x W^T: x rounded to 8-bit integers with a scale per row
               (amax / 127), W integers with a scale per output channel

Each case is made from a seed; ``run`` is one pass, in elementary torch
operations, or through the library where ``own`` is set; ``exact`` is the
definition in 64 bits.  Slots without a row keep the zeros that ``prepare`` put
there.
"""
import math

import torch

own = False


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the smallest model: a few rows for each of 16 experts, nothing but latency
        dict(name="ffn_tiny", op="ffn", fmt="bf16", N=128, K=2, E=16, share=1, A=1, H=256, I=128),
        # a decode batch over the 32 experts of one of eight GPUs: about 16 rows an
        # expert, the weights are the bytes that count
        dict(name="ffn_decode", op="ffn", fmt="bf16", N=64, K=8, E=32, share=1, A=1, H=7168,
             I=2048),
        # what a prefill batch of 4096 tokens sends to these experts: about 128 rows each
        dict(name="ffn_rank", op="ffn", fmt="bf16", N=512, K=8, E=32, share=1, A=128, H=7168,
             I=2048),
        # the expert that every token passes: one plain matrix of rows
        dict(name="ffn_shared", op="ffn", fmt="bf16", N=4096, K=1, E=0, share=1, A=1, H=7168,
             I=2048),
        # the same experts' rows with 8-bit integer weights
        dict(name="ffn_rank_int8", op="ffn", fmt="int8", N=512, K=8, E=32, share=1, A=128, H=7168,
             I=2048),
        # training: odd sizes, uneven counts, part of the choices elsewhere
        dict(name="grad_ragged", op="ffn_grad", N=701, K=3, E=12, share=2, A=16, H=1000, I=344),
        # training: 512 rows an expert
        dict(name="grad_rank", op="ffn_grad", N=1024, K=8, E=16, share=1, A=128, H=7168, I=2048),
        # combine's gradient: a decode-sized batch, then the prefill batch
        dict(name="combine_grad_decode", op="combine_grad", N=128, K=8, E=256, share=1, A=1,
             H=7168),
        dict(name="combine_grad_prefill", op="combine_grad", N=4096, K=8, E=256, share=1, A=128,
             H=7168),
        # a projection of one token
        dict(name="int8_one", op="int8", N=1, K=1, E=0, share=1, A=1, C=7168, O=7168),
        # odd sizes, grouped over experts
        dict(name="int8_ragged", op="int8", N=93, K=3, E=10, share=2, A=4, C=2000, O=1237),
        # a projection of the prefill batch
        dict(name="int8_prefill", op="int8", N=4096, K=1, E=0, share=1, A=1, C=7168, O=7168),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("ffn", "ffn", "ffn_grad", "combine_grad", "int8"))
    fmt = rng.choice(("bf16", "int8")) if op == "ffn" else "int8" if op == "int8" else "bf16"
    unit = 16 if fmt == "int8" else 8
    size = lambda lo, hi: _log(rng, lo // unit, hi // unit) * unit      # noqa: E731
    if op == "combine_grad":
        return dict(op=op, N=_log(rng, 1, 4096), K=rng.randint(1, 10), E=_log(rng, 16, 256),
                    share=rng.choice((1, 1, 2)), A=rng.choice((1, 16, 128)), H=size(64, 7168))
    E = rng.choice((0, _log(rng, 1, 32)))
    K = rng.randint(1, min(8, E)) if E else 1
    c = dict(op=op, N=_log(rng, 1, 4096 // K), K=K, E=E,
             share=rng.choice((1, 1, 2)) if E else 1, A=rng.choice((1, 16, 128)))
    if c["N"] * K < 16 * c["share"]:       # some choices have to stay on this GPU
        c["share"] = 1
    if op == "int8":
        return dict(c, C=size(64, 7168), O=_log(rng, 50, 4096))
    c.update(H=size(64, 4096), I=size(32, 1536))
    return dict(c, fmt=fmt) if op == "ffn" else c


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape, scale=1.0):
    """bf16 values of N(0, scale^2), a matrix at a time."""
    t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for m in (t if len(shape) == 3 else [t]):
        m.copy_(torch.randn(m.shape, generator=gen, device="cuda") * scale)
    return t


def _int8_weight(gen, *shape):
    """Codes as a quantised N(0, 1 / cols) weight has them, and their scales."""
    q = torch.empty(shape, dtype=torch.int8, device="cuda")
    for m in (q if len(shape) == 3 else [q]):
        m.copy_((torch.randn(m.shape, generator=gen, device="cuda") * 36).round_()
                .clamp_(-127, 127))
    s = (torch.rand(shape[:-1], generator=gen, device="cuda") + 0.5) * shape[-1] ** -0.5 / 36
    return q, s


def _routing(c, gen, st):
    """Choices of distinct experts, some more popular; the slots of the pairs as the
    routing layout numbers them; for each expert the slots of its rows."""
    N, K, E, A = c["N"], c["K"], c["E"], c["A"]
    total = E * c["share"]
    likes = torch.randn((total,), generator=gen, device="cuda") * 0.3
    noise = -torch.log(-torch.log(torch.rand((N, total), generator=gen, device="cuda")
                                  .clamp(1e-6, 1 - 1e-6)))
    idx = torch.sort(likes + noise, dim=1, descending=True)[1][:, :K]
    idx = torch.where(idx < E, idx, torch.full_like(idx, -1))
    flat = idx.reshape(-1)
    order = torch.sort(torch.where(flat < 0, torch.full_like(flat, E), flat), stable=True)[1]
    count = torch.bincount(flat + 1, minlength=E + 1)[1:]
    ends = ((count + A - 1) // A * A).cumsum(0)
    off = ends - (count + A - 1) // A * A
    held = int(count.sum())
    by = flat[order[:held]]
    slot = off[by] + torch.arange(held, device="cuda") - (count.cumsum(0) - count)[by]
    slot_of = torch.full_like(flat, -1)
    slot_of[order[:held]] = slot
    cap = N * K + E * (A - 1)
    most = max(1, int(count.max()))
    pos = torch.arange(most, device="cuda")
    ok = pos < count[:, None]
    rows = torch.where(ok, off[:, None] + pos, torch.zeros_like(off)[:, None])
    back = torch.full((cap,), E * most, device="cuda")        # slot -> its place in [E, most]
    back[slot] = by * most + slot - off[by]
    st.update(idx=idx.to(torch.int32), slot_of=slot_of.view(N, K), count=count, off=off, cap=cap,
              rows=rows, ok=ok, back=back)
    if own:
        import combine_ep_get_amd as ep
        st["layout"] = ep.get_layout(st["idx"], E, 1, A)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c = dict(case)
    st = dict(case=c, layout=None, cap=c["N"])
    if c["E"]:
        _routing(c, gen, st)
    cap, lead = st["cap"], (c["E"],) if c["E"] else ()
    zeros = lambda cols: torch.zeros((cap, cols), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    if c["op"] == "combine_grad":
        st["eo"] = _normal(gen, cap, c["H"])
        st["dy"] = _normal(gen, c["N"], c["H"])
        g = torch.rand(st["slot_of"].shape, generator=gen, device="cuda") + 0.2
        st["wts"] = g / g.sum(dim=1, keepdim=True)
        st["deo"] = zeros(c["H"])
        st["dwts"] = torch.empty_like(st["wts"])
        return st
    if c["op"] == "int8":
        st["x"] = _normal(gen, cap, c["C"])
        st["w"] = _int8_weight(gen, *lead, c["O"], c["C"])
        st["y"] = zeros(c["O"])
        if own:
            import combine_ep_get_amd as ep
            st["handle"] = ep.Int8Weight(*st["w"])
        return st
    H, I = c["H"], c["I"]
    st["x"] = _normal(gen, cap, H)
    if c.get("fmt") == "int8":
        st["w13"], st["w2"] = _int8_weight(gen, *lead, 2 * I, H), _int8_weight(gen, *lead, H, I)
    else:
        st["w13"] = _normal(gen, *lead, 2 * I, H, scale=H ** -0.5)
        st["w2"] = _normal(gen, *lead, H, I, scale=I ** -0.5)
    st["y"] = zeros(H)                 # y, or the gradient of x
    if c["op"] == "ffn_grad":
        st["gu"] = _normal(gen, cap, 2 * I)
        st["dy"] = _normal(gen, cap, H)
        st["dw13"], st["dw2"] = torch.empty_like(st["w13"]), torch.empty_like(st["w2"])
    if own:
        import combine_ep_get_amd as ep
        st["ws"] = ep.alloc_ffn_workspace(cap, H, I, int8=c.get("fmt") == "int8",
                                          backward=c["op"] == "ffn_grad")
        if c.get("fmt") == "int8":
            st["h13"], st["h2"] = ep.Int8Weight(*st["w13"]), ep.Int8Weight(*st["w2"])
        else:
            st["h13"], st["h2"] = st["w13"], st["w2"]
    return st


# ------------------------------------------------------------------ plain forms
def _by_expert(st, t):
    """Rows in 32 bits as [experts, rows, cols], zeros behind an expert's last."""
    if not st["case"]["E"]:
        return t.float()[None]
    return t[st["rows"]].float() * st["ok"][:, :, None]


def _to_slots(st, p, out):
    """The inverse: rounds to out's type, zeros where a slot has no row."""
    if not st["case"]["E"]:
        return out.copy_(p[0])
    p = torch.cat([p.reshape(-1, p.shape[-1]), p.new_zeros((1, p.shape[-1]))])
    return out.copy_(p[st["back"]])


def _stack(w):
    """A weight in 32 bits, [experts, rows, cols]."""
    if not isinstance(w, tuple):
        return w.float() if w.dim() == 3 else w.float()[None]
    q = w[0].float()
    return q if q.dim() == 3 else q[None]


def _channels(w):
    return w[1][..., None, :] if w[1].dim() == 2 else w[1][None, None]


def _round_rows(x):
    """Whole numbers of each row, and its scale: amax / 127, rounded once to 32 bits
    (1 for a row of zeros); a quotient next to a half is decided in 64 bits."""
    scale = (x.abs().amax(dim=-1, keepdim=True).double() / 127).float()
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    return (x.double() / scale.double()).round().clamp(-127, 127).float(), scale


def _product(x, w):
    """x W^T of each expert."""
    if isinstance(w, tuple):
        q, scale = _round_rows(x)
        return torch.matmul(q, _stack(w).transpose(1, 2)) * scale * _channels(w)
    return torch.matmul(x, _stack(w).transpose(1, 2))


def _plain_ffn(st):
    I = st["case"]["I"]
    both = _product(_by_expert(st, st["x"]), st["w13"])
    g, u = both[..., :I], both[..., I:]
    hidden = g / (1 + torch.exp(-g)) * u
    if st["case"]["fmt"] == "int8":    # by definition the codes are those of bf16 rows
        hidden = hidden.to(torch.bfloat16).float()
    return _to_slots(st, _product(hidden, st["w2"]), st["y"])


def _plain_ffn_grad(st):
    I = st["case"]["I"]
    x, dy, gu = (_by_expert(st, st[k]) for k in ("x", "dy", "gu"))
    w13, w2 = _stack(st["w13"]), _stack(st["w2"])
    g, u = gu[..., :I], gu[..., I:]
    sig = 1 / (1 + torch.exp(-g))
    dh = torch.matmul(dy, w2)
    dgu = torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], dim=2)
    dx = _to_slots(st, torch.matmul(dgu, w13), st["y"])
    st["dw13"].copy_(torch.matmul(dgu.transpose(1, 2), x).view_as(st["dw13"]))
    st["dw2"].copy_(torch.matmul(dy.transpose(1, 2), g * sig * u).view_as(st["dw2"]))
    return dx, st["dw13"], st["dw2"]


def _plain_combine_grad(st):
    slot, dy = st["slot_of"], st["dy"].float()[:, None]
    has = slot >= 0
    eo = st["eo"][slot.clamp(min=0)].float()
    dwts = (eo * dy).sum(dim=2) * has
    pairs = torch.where(has, slot, torch.full_like(slot, st["cap"])).view(-1)
    deo = torch.zeros((st["cap"] + 1, dy.shape[2]), dtype=torch.bfloat16, device=dy.device)
    deo[pairs] = (st["wts"][:, :, None] * dy).view(-1, dy.shape[2]).to(torch.bfloat16)
    return deo[:-1], dwts


def run(state):
    c = state["case"]
    if not own:
        if c["op"] == "ffn":
            return _plain_ffn(state)
        if c["op"] == "ffn_grad":
            return _plain_ffn_grad(state)
        if c["op"] == "combine_grad":
            return _plain_combine_grad(state)
        return _to_slots(state, _product(_by_expert(state, state["x"]), state["w"]), state["y"])
    import combine_ep_get_amd as ep
    if c["op"] == "ffn":
        return ep.expert_ffn(state["x"], state["h13"], state["h2"], layout=state["layout"],
                             out=state["y"], workspace=state["ws"])
    if c["op"] == "ffn_grad":
        return ep.expert_ffn_backward(state["dy"], state["x"], state["gu"], state["h13"],
                                      state["h2"], layout=state["layout"],
                                      out=(state["y"], state["dw13"], state["dw2"]),
                                      workspace=state["ws"])
    if c["op"] == "combine_grad":
        return ep.combine_backward(state["dy"], state["eo"], state["layout"], state["wts"],
                                   out=(state["deo"], state["dwts"]))
    return ep.int8_linear(state["x"], state["handle"], layout=state["layout"], out=state["y"])


# ------------------------------------------------------------------ costs
def work(case):
    c = case
    E, rows = c["E"], c["N"] * c["K"] / c["share"]
    # experts that at least one token names, on average over even routings
    active = E * (1 - (1 - c["K"] / (E * c["share"])) ** c["N"]) if E else 1
    if c["op"] == "combine_grad":
        return {"bytes": 2 * c["H"] * (c["N"] + 2 * rows) + 12 * c["N"] * c["K"],
                "flops": 3 * rows * c["H"]}
    if c["op"] == "int8":
        return {"bytes": active * c["O"] * (c["C"] + 4) + 2 * rows * (c["C"] + c["O"]),
                "flops": 2 * rows * c["C"] * c["O"]}
    H, I = c["H"], c["I"]
    if c["op"] == "ffn":
        weight = 3 * H * I + 4 * (2 * I + H) if c["fmt"] == "int8" else 6 * H * I
        return {"bytes": active * weight + 4 * rows * H, "flops": 6 * rows * H * I}
    return {"bytes": (active + max(E, 1)) * 6 * H * I + rows * (6 * H + 4 * I),
            "flops": 12 * rows * H * I}


# ------------------------------------------------------------------ the definition in 64 bits
def _experts(st):
    """(expert or None, its slots) one after the other."""
    if not st["case"]["E"]:
        return [(None, slice(0, st["case"]["N"]))]
    at = zip(st["off"].tolist(), st["count"].tolist())
    return [(e, slice(o, o + n)) for e, (o, n) in enumerate(at)]


def _mm8(x, w, e):
    """x W^T as the sums of 8-bit codes times both scales, x [rows, cols] in 64 bits."""
    pick = (lambda t: t) if e is None else (lambda t: t[e])
    amax = x.abs().max(dim=1)[0]
    step = torch.where(amax > 0, amax / 127.0, torch.ones_like(amax)).float().double()
    codes = torch.clamp(torch.round(x / step[:, None]), -127.0, 127.0)
    sums = torch.mm(codes, pick(w[0]).double().t())
    return sums * torch.outer(step, pick(w[1]).double())


def exact(case, seed):
    st = prepare(case, seed)
    op, I = case["op"], case.get("I")
    dev = dict(dtype=torch.float64, device="cuda")
    if op == "combine_grad":
        deo = torch.zeros((st["cap"], case["H"]), **dev)
        dwts = torch.zeros((case["N"], case["K"]), **dev)
        dy = st["dy"].double()
        for k in range(case["K"]):
            t = (st["slot_of"][:, k] >= 0).nonzero()[:, 0]
            s = st["slot_of"][t, k]
            dwts[t, k] = torch.einsum("th,th->t", st["eo"][s].double(), dy[t])
            deo[s] = st["wts"][t, k].double()[:, None] * dy[t]
        return deo, dwts
    y = torch.zeros(st["y"].shape, **dev)
    if op == "ffn_grad":
        dw13, dw2 = torch.zeros(st["w13"].shape, **dev), torch.zeros(st["w2"].shape, **dev)
    for e, at in _experts(st):
        x = st["x"][at].double()
        if x.shape[0] == 0:
            continue
        if op == "int8":
            y[at] = _mm8(x, st["w"], e)
        elif op == "ffn" and case["fmt"] == "int8":
            both = _mm8(x, st["w13"], e)
            h = both[:, I:] * both[:, :I] * torch.sigmoid(both[:, :I])
            y[at] = _mm8(h.to(torch.bfloat16).double(), st["w2"], e)
        else:
            w13, w2 = ((st[k] if e is None else st[k][e]).double() for k in ("w13", "w2"))
            if op == "ffn":
                both = torch.mm(x, w13.t())
                y[at] = torch.mm(both[:, I:] * both[:, :I] * torch.sigmoid(both[:, :I]), w2.t())
                continue
            dy, g, u = st["dy"][at].double(), st["gu"][at, :I].double(), st["gu"][at, I:].double()
            s = torch.sigmoid(g)
            dh = torch.mm(dy, w2)
            dgu = torch.cat([dh * u * (s + g * s * (1 - s)), dh * (g * s)], dim=1)
            y[at] = torch.mm(dgu, w13)
            (dw13 if e is None else dw13[e]).copy_(torch.mm(dgu.t(), x))
            (dw2 if e is None else dw2[e]).copy_(torch.mm(dy.t(), g * s * u))
    return (y, dw13, dw2) if op == "ffn_grad" else y
