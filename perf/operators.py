"""The expert-layer operators at the sizes they are used at.

Three operators that stand between the routing layout and the model: the router
(``route``: gate logits to expert ids and weights), the whole expert layer for
a few tokens (``moe_layer``: both expert products, the gate and the weighted
sum, without dispatch and combine) and the product of a few rows with a 4-bit
weight matrix (``quant_linear``).  Each case is made from a seed; ``run`` is one
pass, in elementary torch operations, or through the library where ``own`` is
set; ``exact`` is the definition in 64 bits.

4-bit weights, ``codes`` uint8 [..., rows, cols/2]:
  int4   value = scale[row, group] * (code - zero), zero 8 where no zeros are
         given; group 32, 64 or 128 columns, scale bf16.  The eight nibbles of
         a little-endian 32-bit word, lowest first, hold columns
         0, 2, 4, 6, 1, 3, 5, 7 of their block of eight.
  mxfp4  OCP MX: E2M1 codes (sign in bit 3), lower nibble first, times
         2^(scale - 127) per 32 columns, scale uint8.
"""
import math

import torch

own = False

NIBBLE_COLUMNS = (0, 2, 4, 6, 1, 3, 5, 7)      # int4: column that nibble j holds
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases
def listed():
    big = dict(H=7168, I=2048, E=32, K=8)
    return [
        # one token of a decode step through a gate with bias-corrected,
        # group-limited selection: nothing but latency
        dict(name="route_one", op="route", N=1, E=256, K=8, dtype="float32", scoring="sigmoid",
             bias=True, groups=8, topk_groups=4, group_top=2, renorm=True, scale=2.5),
        # the prefill batch with the same gate
        dict(name="route_prefill", op="route", N=4096, E=256, K=8, dtype="float32",
             scoring="sigmoid", bias=True, groups=8, topk_groups=4, group_top=2, renorm=True,
             scale=2.5),
        # the largest batch, a plain softmax gate on bf16 logits (many ties)
        dict(name="route_large", op="route", N=16384, E=256, K=8, dtype="bfloat16",
             scoring="softmax", bias=False, groups=1, topk_groups=1, group_top=1, renorm=True,
             scale=1.0),
        # the smallest model: two launches with almost no work
        dict(name="moe_tiny_bf16", op="moe", N=16, H=256, I=128, E=16, K=2, share=1, fmt="bf16",
             group=0, zeros=False),
        # one token of a decode step, its eight experts all on this GPU
        dict(name="moe_one_bf16", op="moe", N=1, share=1, fmt="bf16", group=0, zeros=False, **big),
        # a decode batch on a GPU that holds 32 of 256 experts: most choices
        # belong elsewhere (-1)
        dict(name="moe_rank_bf16", op="moe", N=256, share=8, fmt="bf16", group=0, zeros=False,
             **big),
        # the single token again with 4-bit experts
        dict(name="moe_one_int4", op="moe", N=1, share=1, fmt="int4", group=128, zeros=False,
             **big),
        # 64 tokens, every expert with about 16 of them
        dict(name="moe_batch_int4", op="moe", N=64, share=1, fmt="int4", group=128, zeros=False,
             **big),
        # odd sizes, part of the choices elsewhere
        dict(name="moe_ragged_mxfp4", op="moe", N=13, H=1952, I=992, E=24, K=5, share=2,
             fmt="mxfp4", group=32, zeros=False),
        # a dense projection of one token
        dict(name="linear_one_int4", op="linear", N=1, O=7168, C=7168, fmt="int4", group=128,
             zeros=False),
        # a small decode batch, odd row count
        dict(name="linear_ragged_mxfp4", op="linear", N=11, O=1237, C=2016, fmt="mxfp4", group=32,
             zeros=False),
        # a larger batch with zero points and finer groups
        dict(name="linear_batch_int4", op="linear", N=64, O=7168, C=2048, fmt="int4", group=64,
             zeros=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "moe", "moe", "linear"))
    if op == "route":
        groups = rng.choice((1, 1, 4, 8))
        per = _log(rng, 4, 512 // groups)
        E = groups * per
        N = min(_log(rng, 1, 16384), 16384 * 256 // E)
        tg = rng.randint(1, groups)
        return dict(op=op, N=N, E=E, K=rng.randint(1, min(16, tg * per)),
                    dtype=rng.choice(("float32", "bfloat16")),
                    scoring=rng.choice(("sigmoid", "softmax")), bias=rng.random() < 0.5,
                    groups=groups, topk_groups=tg,
                    group_top=rng.choice((1, 2)) if groups > 1 else 1,
                    renorm=rng.random() < 0.8, scale=rng.choice((1.0, 2.5)))
    fmt = rng.choice(("bf16", "int4", "mxfp4") if op == "moe" else ("int4", "mxfp4"))
    group = {"bf16": 0, "mxfp4": 32, "int4": rng.choice((32, 64, 128, 128))}[fmt]
    unit = group or 8
    zeros = fmt == "int4" and rng.random() < 0.3
    cols = lambda lo, hi: max(1, _log(rng, lo, hi) // unit) * unit      # noqa: E731
    if op == "linear":
        return dict(op=op, N=_log(rng, 1, 64), O=_log(rng, 64, 8192), C=cols(256, 7168), fmt=fmt,
                    group=group, zeros=zeros)
    N, K = _log(rng, 1, 64 if fmt == "int4" else 128), rng.randint(1, 8)
    share = rng.choice((1, 1, 2, 8))
    if N * K < 16 * share:             # some choices have to stay on this GPU
        share = 1
    return dict(op=op, N=N, H=cols(256, 4096),
                I=cols(64, 1024), E=max(_log(rng, 4, 64), -(-K // share)), K=K, share=share,
                fmt=fmt, group=group, zeros=zeros)


# ------------------------------------------------------------------ inputs
def _codes(fmt, rows, cols, gen):
    """Codes as a quantised N(0, 1) weight has them, one per byte, in column order."""
    v = torch.randn((rows, cols), generator=gen, device="cuda")
    if fmt == "int4":
        return ((v * 2.2).round_().clamp_(-8, 7) + 8).to(torch.uint8)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    return (torch.bucketize((v * 2).abs(), edges) + 8 * (v < 0)).to(torch.uint8)


def _pack(fmt, c):
    c = c.view(c.shape[0], -1, 8)
    order = NIBBLE_COLUMNS if fmt == "int4" else tuple(range(8))
    return torch.stack([c[:, :, order[2 * b]] | (c[:, :, order[2 * b + 1]] << 4)
                        for b in range(4)], dim=2).view(c.shape[0], -1)


def _weight(fmt, lead, rows, cols, group, zeros, gen):
    """A weight [*lead, rows, cols] whose products with N(0, 1) rows are about N(0, 1)."""
    n = math.prod(lead)
    if fmt == "bf16":
        w = torch.empty((n, rows, cols), dtype=torch.bfloat16, device="cuda")
        for e in range(n):
            w[e] = torch.randn((rows, cols), generator=gen, device="cuda") * cols ** -0.5
        return dict(fmt=fmt, w=w.view(*lead, rows, cols))
    codes = torch.empty((n, rows, cols // 2), dtype=torch.uint8, device="cuda")
    for e in range(n):
        codes[e] = _pack(fmt, _codes(fmt, rows, cols, gen))
    G = cols // group
    if fmt == "int4":
        s = (torch.rand((n, rows, G), generator=gen, device="cuda") + 0.5) * cols ** -0.5 / 2.2
        s = s.to(torch.bfloat16)
    else:
        s = torch.randint(-1, 2, (n, rows, G), generator=gen, device="cuda")
        s = (s + (126 - round(0.5 * math.log2(cols)))).to(torch.uint8)
    z = None
    if zeros:
        z = torch.randint(6, 11, (n, rows, G), generator=gen, device="cuda").to(torch.uint8)
        z = z.view(*lead, rows, G)
    return dict(fmt=fmt, w=codes.view(*lead, rows, cols // 2), s=s.view(*lead, rows, G), z=z,
                group=group)


def _handle(ep, w):
    if w["fmt"] == "bf16":
        return w["w"]
    return ep.QuantWeight(w["w"], w["s"], zeros=w["z"], group=w["group"], fmt=w["fmt"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c = dict(case)
    st = dict(case=c)
    if c["op"] == "route":
        l = 1.5 * torch.randn((c["N"], c["E"]), generator=gen, device="cuda")
        st["logits"] = l.to(getattr(torch, c["dtype"]))
        st["bias"] = (0.1 * torch.randn((c["E"],), generator=gen, device="cuda")
                      if c["bias"] else None)
        return st
    if c["op"] == "linear":
        st["x"] = torch.randn((c["N"], c["C"]), generator=gen, device="cuda").to(torch.bfloat16)
        st["w"] = _weight(c["fmt"], (), c["O"], c["C"], c["group"], c["zeros"], gen)
        if own:
            import combine_ep_get_amd as ep
            st["handle"] = _handle(ep, st["w"])
        return st
    N, H, I, E, K = c["N"], c["H"], c["I"], c["E"], c["K"]
    st["x"] = torch.randn((N, H), generator=gen, device="cuda").to(torch.bfloat16)
    scores = torch.rand((N, E * c["share"]), generator=gen, device="cuda")
    idx = torch.sort(scores, dim=1, descending=True)[1][:, :K].to(torch.int32)
    st["idx"] = torch.where(idx < E, idx, torch.full_like(idx, -1))
    g = torch.rand((N, K), generator=gen, device="cuda") + 0.2
    st["wts"] = g / g.sum(dim=1, keepdim=True)
    st["w13"] = _weight(c["fmt"], (E,), 2 * I, H, c["group"], c["zeros"], gen)
    st["w2"] = _weight(c["fmt"], (E,), H, I, c["group"], c["zeros"], gen)
    if own:
        import combine_ep_get_amd as ep
        st["h13"], st["h2"] = _handle(ep, st["w13"]), _handle(ep, st["w2"])
        st["y"] = torch.empty_like(st["x"])
        st["ws"] = ep.alloc_moe_workspace(N, K, E, H, I)
    return st


# ------------------------------------------------------------------ plain forms
def _dense(w, e=None):
    """The weight in 32 bits; of a stack of experts, that of expert e ([1] tensor or int)."""
    pick = (lambda t: t) if e is None else \
        (lambda t: t[e]) if isinstance(e, int) else (lambda t: t.index_select(0, e)[0])
    if w["fmt"] == "bf16":
        return pick(w["w"]).float()
    c = pick(w["w"])
    rows = c.shape[0]
    nib = torch.stack((c & 15, c >> 4), dim=2).view(rows, -1, 8)   # nibble j of each word
    if w["fmt"] == "int4":
        back = [NIBBLE_COLUMNS.index(j) for j in range(8)]
        v = nib[:, :, back].float()
        v = v.reshape(rows, -1, w["group"])
        zero = 8.0 if w["z"] is None else pick(w["z"]).float()[:, :, None]
        return ((v - zero) * pick(w["s"]).float()[:, :, None]).view(rows, -1)
    m, ex, neg = (nib & 1).float(), ((nib >> 1) & 3).float(), (nib >> 3).float()
    v = torch.where(ex == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(ex - 1)) * (1 - 2 * neg)
    return (v.reshape(rows, -1, 32) * torch.exp2(pick(w["s"]).float() - 127)[:, :, None]) \
        .view(rows, -1)


def _plain_route(st):
    c = st["case"]
    N, E, K, G = c["N"], c["E"], c["K"], c["groups"]
    l = st["logits"].double()          # neighbours at the border differ by less than 2^-24
    if c["scoring"] == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
    else:
        s = torch.exp(l - l.max(dim=1, keepdim=True)[0])
        s = s / s.sum(dim=1, keepdim=True)
    value = s if st["bias"] is None else s + st["bias"].double()
    order = l if st["bias"] is None else value       # the scores grow with the logits
    if G > 1:
        best = torch.sort(value.view(N, G, -1), dim=2, descending=True)[0]
        best = best[:, :, :c["group_top"]].sum(dim=2)
        kept = torch.sort(best, dim=1, descending=True, stable=True)[1][:, :c["topk_groups"]]
        keep = torch.zeros((N, G), dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        keep = keep[:, :, None].expand(N, G, E // G).reshape(N, E)
        order = torch.where(keep, order, torch.full_like(order, -math.inf))
    idx = torch.sort(order, dim=1, descending=True, stable=True)[1][:, :K]
    w = s.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return idx.to(torch.int32), (w * c["scale"]).float()


def _plain_moe(st):
    c = st["case"]
    N, I, E, K = c["N"], c["I"], c["E"], c["K"]
    x, idx = st["x"].float(), st["idx"]
    wts = torch.where(idx >= 0, st["wts"], torch.zeros_like(st["wts"]))
    y = torch.zeros_like(x)

    def expert(rows, e):
        gu = rows @ _dense(st["w13"], e).t()
        g, u = gu[:, :I], gu[:, I:]
        return (g / (1 + torch.exp(-g)) * u) @ _dense(st["w2"], e).t()
    if N * K < E:
        for t in range(N):
            for k in range(K):
                e = idx[t, k].clamp(min=0).view(1)
                y[t] += wts[t, k] * expert(x[t:t + 1], e)[0]
    else:
        for e in range(E):
            y += (wts * (idx == e)).sum(dim=1)[:, None] * expert(x, e)
    return y.to(torch.bfloat16)


def run(state):
    c = state["case"]
    if not own:
        if c["op"] == "route":
            return _plain_route(state)
        if c["op"] == "linear":
            return (state["x"].float() @ _dense(state["w"]).t()).to(torch.bfloat16)
        return _plain_moe(state)
    import combine_ep_get_amd as ep
    if c["op"] == "route":
        return ep.route(state["logits"], c["K"], bias=state["bias"], scoring=c["scoring"],
                        num_groups=c["groups"], topk_groups=c["topk_groups"],
                        group_top=c["group_top"], renormalize=c["renorm"], scale=c["scale"])
    if c["op"] == "linear":
        return ep.quant_linear(state["x"], state["handle"])
    return ep.moe_layer(state["x"], state["idx"], state["wts"], state["h13"], state["h2"],
                        out=state["y"], workspace=state["ws"])


# ------------------------------------------------------------------ costs
def _weight_bytes(c, rows, cols):
    if c["fmt"] == "bf16":
        return 2.0 * rows * cols
    G = cols // c["group"]
    return rows * (cols / 2 + G * ((2 if c["fmt"] == "int4" else 1) + (1 if c["zeros"] else 0)))


def work(case):
    c = case
    if c["op"] == "route":
        size = 4 if c["dtype"] == "float32" else 2
        return {"bytes": c["N"] * (c["E"] * size + c["K"] * 8) + (4 * c["E"] if c["bias"] else 0),
                "flops": 8.0 * c["N"] * c["E"]}
    if c["op"] == "linear":
        return {"bytes": _weight_bytes(c, c["O"], c["C"]) + 2 * c["N"] * (c["O"] + c["C"]),
                "flops": 2.0 * c["N"] * c["O"] * c["C"]}
    N, H, I, E, K = c["N"], c["H"], c["I"], c["E"], c["K"]
    # experts that at least one token names, on average over the routings
    active = E * (1 - (1 - K / (E * c["share"])) ** N)
    return {"bytes": active * (_weight_bytes(c, 2 * I, H) + _weight_bytes(c, H, I))
            + N * (4 * H + 8 * K),
            "flops": 6.0 * N * K / c["share"] * H * I}


# ------------------------------------------------------------------ the definition in 64 bits
def _table64(w, e=None):
    """The weight in 64 bits, each code looked up in the table of its format."""
    at = (lambda t: t) if e is None else (lambda t: t[e])
    if w["fmt"] == "bf16":
        return at(w["w"]).double()
    codes = at(w["w"]).to(torch.int64)
    rows, cols = codes.shape[0], 2 * codes.shape[1]
    table = range(16) if w["fmt"] == "int4" else E2M1 + tuple(-v for v in E2M1)
    table = torch.tensor([float(v) for v in table], dtype=torch.float64, device=codes.device)
    out = torch.empty((rows, cols), dtype=torch.float64, device=codes.device)
    for j in range(8):                 # nibble j of every word of four bytes
        col = NIBBLE_COLUMNS[j] if w["fmt"] == "int4" else j
        out[:, col::8] = table[(codes[:, j // 2::4] >> (4 * (j % 2))) & 15]
    grouped = out.view(rows, -1, w["group"])
    if w["fmt"] == "int4":
        grouped -= 8.0 if w["z"] is None else at(w["z"]).double().unsqueeze(2)
        grouped *= at(w["s"]).double().unsqueeze(2)
    else:
        grouped *= torch.pow(torch.tensor(2.0, dtype=torch.float64, device=codes.device),
                             at(w["s"]).double() - 127).unsqueeze(2)
    return out


def _exact_route(st):
    import numpy as np
    c = st["case"]
    l = st["logits"].double().cpu().numpy()
    N, E = l.shape
    if c["scoring"] == "sigmoid":
        s = np.where(l >= 0, 1, np.exp(-np.abs(l))) / (1 + np.exp(-np.abs(l)))
    else:
        s = np.exp(l - l.max(1)[:, None])
        s = s / s.sum(1)[:, None]
    v, by = s, l
    if st["bias"] is not None:
        v = by = s + st["bias"].double().cpu().numpy()
    per = E // c["groups"]
    allowed = np.ones((N, c["groups"]), bool)
    if c["groups"] > 1:
        top = -np.partition(-v.reshape(N, -1, per), c["group_top"] - 1, axis=2)
        first = np.argsort(-top[:, :, :c["group_top"]].sum(2), axis=1, kind="stable")
        allowed[:] = False
        np.put_along_axis(allowed, first[:, :c["topk_groups"]], True, axis=1)
    by = np.where(np.repeat(allowed, per, axis=1), by, -np.inf)
    idx = np.argsort(-by, axis=1, kind="stable")[:, :c["K"]]
    w = np.take_along_axis(s, idx, axis=1)
    if c["renorm"]:
        w = w / w.sum(1)[:, None]
    return torch.from_numpy(idx.astype(np.int32)), torch.from_numpy(w * c["scale"])


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(st)
    if case["op"] == "linear":
        return torch.mm(st["x"].double(), _table64(st["w"]).t())
    I = case["I"]
    x, idx, wts = st["x"].double(), st["idx"].cpu(), st["wts"].double()
    y = torch.zeros_like(x)
    for e in range(case["E"]):
        pairs = [(t, k) for t, k in (idx == e).nonzero().tolist()]
        if not pairs:
            continue
        tok = torch.tensor([t for t, _ in pairs], device=x.device)
        gate = torch.stack([wts[t, k] for t, k in pairs])
        both = torch.mm(_table64(st["w13"], e), x[tok].t())
        hidden = both[I:] * both[:I] * torch.sigmoid(both[:I])
        y.index_add_(0, tok, torch.mm(_table64(st["w2"], e), hidden).t() * gate[:, None])
    return y
