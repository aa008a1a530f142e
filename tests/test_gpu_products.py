"""The expert layer for a few tokens and the 4-bit product on the GPU, against
plain 64-bit implementations with bounds from the arithmetic (product_ref.py)."""
import copy

import pytest
import torch

import combine_ep_get_amd as ep
from tests import product_ref as ref

pytestmark = pytest.mark.gpu


def inputs(N, H, E, K, gen, absent=0.2):
    x = torch.randn((N, H), generator=gen).to(torch.bfloat16)
    idx = torch.randint(0, E, (N, K), generator=gen, dtype=torch.int32)
    idx[torch.rand((N, K), generator=gen) < absent] = -1
    return x, idx, torch.rand((N, K), generator=gen) + 0.1


def held(y, want, bound):
    y = y.double().cpu()
    off = (y - want).abs() - bound
    assert torch.isfinite(y).all()
    assert (off <= 0).all(), f"{int((off > 0).sum())} values outside, worst {float(off.max())}"


def layer(x, idx, wts, w13, w2, **kw):
    return ep.moe_layer(x.cuda(), idx.cuda(), wts.cuda(), w13.arg, w2.arg, **kw)


FORMATS = [("bf16", None, False), ("int4", 128, False), ("int4", 64, False), ("int4", 32, False),
           ("int4", 128, True), ("int4", 64, True), ("int4", 32, True), ("mxfp4", 32, False)]


@pytest.mark.parametrize("fmt,group,zeros", FORMATS[1:])
@pytest.mark.parametrize("N", [1, 3, 4, 5, 16, 17, 33])
def test_linear(fmt, group, zeros, N):
    for rows, steps in ((1, 1), (16, 2), (37, 5), (100, 9)):
        gen = torch.Generator().manual_seed(rows * 100 + N)
        w = ref.W(fmt, (), rows, steps * group, group, zeros, gen)
        x = torch.randn((N, w.cols), generator=gen).to(torch.bfloat16)
        held(ep.quant_linear(x.cuda(), w.arg), *ref.linear(x, w))


@pytest.mark.parametrize("fmt,group", [("int4", 128), ("mxfp4", 32)])
@pytest.mark.parametrize("N,rows,cols", [(256, 129, 384), (64, 300, 2048), (1, 4099, 7168)])
def test_linear_large(fmt, group, N, rows, cols):
    gen = torch.Generator().manual_seed(N)
    w = ref.W(fmt, (), rows, cols, group, False, gen)
    x = torch.randn((N, cols), generator=gen).to(torch.bfloat16)
    y = torch.full((N, rows), 7.0, dtype=torch.bfloat16, device="cuda")
    assert ep.quant_linear(x.cuda(), w.arg, out=y) is y
    held(y, *ref.linear(x, w))


@pytest.mark.parametrize("fmt,group,zeros", FORMATS[1:])
@pytest.mark.parametrize("N", [2, 9, 30])
def test_scales_anywhere(fmt, group, zeros, N):
    """Long rows, whose scales are loaded 16 bytes at a time, and the same from
    addresses and at lengths where they cannot be."""
    gen = torch.Generator().manual_seed(N)
    rows = 70
    for cols in (2048, 4096, 2048 + 256, 1024 + 128):
        w = ref.W(fmt, (), rows, cols, group, zeros, gen)
        x = torch.randn((N, cols), generator=gen).to(torch.bfloat16)
        y = ep.quant_linear(x.cuda(), w.arg)
        held(y, *ref.linear(x, w))
        shifted = []
        for t, off in ((w.arg.scales, 1), (w.arg.zeros, 3)):
            if t is not None:
                room = torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")[off:]
                t = room.view(t.shape).copy_(t)
            shifted.append(t)
        v = ep.QuantWeight(w.arg.codes, shifted[0], zeros=shifted[1], group=group, fmt=fmt)
        held(ep.quant_linear(x.cuda(), v), *ref.linear(x, w))


def test_linear_no_rows():
    w = ref.W("int4", (), 16, 128, gen=torch.Generator().manual_seed(0))
    assert ep.quant_linear(torch.empty((0, 128), dtype=torch.bfloat16, device="cuda"),
                           w.arg).shape == (0, 16)


def test_every_mxfp4_value():
    """All codes under all scales (but NaN, and products beyond float32), exactly."""
    s = torch.arange(255).repeat_interleave(16)
    c = torch.arange(16).repeat(255)
    value = ref.E2M1[c] * torch.pow(torch.tensor(2.0, dtype=torch.float64), s.double() - 127)
    ok = value.abs() < 2.0 ** 128
    s, c, value = s[ok], c[ok], value[ok]
    codes = ep.pack_codes(c.to(torch.uint8)[:, None].expand(-1, 32).contiguous(), "mxfp4")
    w = ep.QuantWeight(codes.cuda(), s.to(torch.uint8)[:, None].cuda(), fmt="mxfp4")
    for n in (1, 5):
        x = torch.zeros((n, 32), dtype=torch.bfloat16)
        x[:, 9] = 1.0
        y = ep.quant_linear(x.cuda(), w).double().cpu()
        normal = value.abs() >= 2.0 ** -126
        assert torch.equal(y[:, normal], value[normal].expand(n, -1))
        assert (y[:, ~normal].abs() <= value[~normal].abs()).all()   # subnormals may flush


def test_every_int4_code_at_every_column():
    cols = 256
    codes = torch.randint(0, 16, (64, cols), generator=torch.Generator().manual_seed(5),
                          dtype=torch.uint8)
    for group in (32, 64, 128):
        s = torch.full((64, cols // group), 0.5, dtype=torch.bfloat16)
        w = ep.QuantWeight(ep.pack_codes(codes).cuda(), s.cuda(), group=group)
        eye = torch.eye(cols, dtype=torch.bfloat16)
        y = ep.quant_linear(eye.cuda(), w).double().cpu()
        assert torch.equal(y, (codes.double().t() - 8) * 0.5)
        y = torch.cat([ep.quant_linear(eye[i:i + 3].contiguous().cuda(), w)
                       for i in range(0, cols, 3)]).double().cpu()
        assert torch.equal(y, (codes.double().t() - 8) * 0.5)


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("N,E,K", [(1, 8, 3), (4, 3, 2), (7, 5, 4), (16, 4, 1), (40, 6, 3)])
def test_layer(fmt, group, zeros, N, E, K):
    gen = torch.Generator().manual_seed(N)
    unit = group or 8
    H, I = (5 * unit, 3 * unit) if unit > 8 else (1000, 136)
    w13 = ref.W(fmt, (E,), 2 * I, H, group, zeros, gen)
    w2 = ref.W(fmt, (E,), H, I, group, zeros, gen)
    x, idx, wts = inputs(N, H, E, K, gen)
    held(layer(x, idx, wts, w13, w2), *ref.moe(x, idx, wts, w13, w2))


@pytest.mark.parametrize("H,I", [(8, 8), (24, 16), (136, 8), (8, 200), (264, 520)])
@pytest.mark.parametrize("N", [1, 6, 20])
def test_layer_small_odd_sizes(H, I, N):
    gen = torch.Generator().manual_seed(H + I + N)
    w13, w2 = ref.W("bf16", (3,), 2 * I, H, gen=gen), ref.W("bf16", (3,), H, I, gen=gen)
    x, idx, wts = inputs(N, H, 3, 2, gen)
    held(layer(x, idx, wts, w13, w2), *ref.moe(x, idx, wts, w13, w2))


@pytest.mark.parametrize("fmt,group", [("bf16", None), ("int4", 128), ("mxfp4", 32)])
@pytest.mark.parametrize("N,n", [(256, 256), (256, 65), (129, 64), (128, 33), (100, 32), (65, 17),
                                 (30, 16), (18, 5), (17, 4)])
def test_layer_many_tokens_of_one_expert(fmt, group, N, n):
    """n of N tokens go to expert 1, a few of the rest to others, most nowhere."""
    gen = torch.Generator().manual_seed(n)
    H, I, E, K = 256, 128, 4, 2
    w13 = ref.W(fmt, (E,), 2 * I, H, group, False, gen)
    w2 = ref.W(fmt, (E,), H, I, group, False, gen)
    x, idx, wts = inputs(N, H, E, K, gen)
    idx[:] = -1
    idx[torch.randperm(N, generator=gen)[:n], 1] = 1
    idx[:5, 0] = torch.tensor([3, 0, 3, 2, 3], dtype=torch.int32)
    held(layer(x, idx, wts, w13, w2), *ref.moe(x, idx, wts, w13, w2))


@pytest.mark.parametrize("fmt,group,zeros,H,I", [
    ("bf16", None, False, 40, 8), ("bf16", None, False, 264, 72), ("mxfp4", 32, False, 32, 32),
    ("mxfp4", 32, False, 288, 160), ("int4", 128, False, 384, 128), ("int4", 32, True, 96, 64)])
@pytest.mark.parametrize("N", [17, 70])
def test_layer_many_experts(fmt, group, zeros, H, I, N):
    """Enough experts for a workgroup on every CU: no contraction is shared out then."""
    gen = torch.Generator().manual_seed(N + I)
    E = 300
    w13 = ref.W(fmt, (E,), 2 * I, H, group, zeros, gen)
    w2 = ref.W(fmt, (E,), H, I, group, zeros, gen)
    x, idx, wts = inputs(N, H, E, 18, gen)
    idx[1] = E - 1                      # the last expert, named by every choice of a token
    idx[: N // 2, 3] = 7
    held(layer(x, idx, wts, w13, w2), *ref.moe(x, idx, wts, w13, w2))


@pytest.mark.parametrize("fmt,group", [("bf16", None), ("int4", 32), ("mxfp4", 32)])
@pytest.mark.parametrize("E", [1024, 40])
def test_layer_most_pairs(fmt, group, E):
    """The largest batch, 32 choices each: of the most experts, and of a few."""
    gen = torch.Generator().manual_seed(E)
    N, H, I, K = 256, 64, 32, 32
    w13 = ref.W(fmt, (E,), 2 * I, H, group, False, gen)
    w2 = ref.W(fmt, (E,), H, I, group, False, gen)
    x, idx, wts = inputs(N, H, E, K, gen, absent=0.0)
    held(layer(x, idx, wts, w13, w2), *ref.moe(x, idx, wts, w13, w2))


def test_layer_in_place():
    for N in (2, 12, 50):
        x, idx, wts, w13, w2 = small(N=N)
        want = layer(x, idx, wts, w13, w2)
        y = x.cuda()
        assert ep.moe_layer(y, idx.cuda(), wts.cuda(), w13.arg, w2.arg, out=y) is y
        assert torch.equal(y, want)


@pytest.mark.parametrize("fmt,group,zeros,H,I", [
    ("mxfp4", 32, False, 512, 160), ("mxfp4", 32, False, 96, 288), ("int4", 32, True, 256, 192),
    ("int4", 128, False, 384, 256), ("int4", 64, False, 512, 192)])
@pytest.mark.parametrize("N", [13, 16])
def test_layer_few_tokens_of_many_experts(fmt, group, zeros, H, I, N):
    """Up to 16 tokens that name most of the experts: the wavefronts share x."""
    gen = torch.Generator().manual_seed(N + H)
    E, K = 260, 30
    w13 = ref.W(fmt, (E,), 2 * I, H, group, zeros, gen)
    w2 = ref.W(fmt, (E,), H, I, group, zeros, gen)
    x, idx, wts = inputs(N, H, E, K, gen)
    idx[0, :2] = E - 1
    held(layer(x, idx, wts, w13, w2), *ref.moe(x, idx, wts, w13, w2))
    clean = layer(x, idx, wts, w13, w2).cpu()
    x[3] = float("nan")                 # stays in its row
    y = layer(x, idx, wts, w13, w2).cpu()
    assert torch.equal(y[4:], clean[4:]) and torch.equal(y[:3], clean[:3])


def small(seed=3, N=9, H=128, I=64, E=6, K=3, fmt="bf16"):
    gen = torch.Generator().manual_seed(seed)
    group = None if fmt == "bf16" else 32
    return (*inputs(N, H, E, K, gen), ref.W(fmt, (E,), 2 * I, H, group, False, gen),
            ref.W(fmt, (E,), H, I, group, False, gen))


def test_layer_no_tokens_no_experts():
    x, idx, wts, w13, w2 = small()
    y = ep.moe_layer(torch.empty((0, 128), dtype=torch.bfloat16, device="cuda"),
                     torch.empty((0, 3), dtype=torch.int32, device="cuda"),
                     torch.empty((0, 3), device="cuda"), w13.arg, w2.arg)
    assert y.shape == (0, 128)
    ws = torch.full((ep.moe_workspace_bytes(0, 3, 6, 128, 64),), 255, dtype=torch.uint8,
                    device="cuda")
    layer(x[:0], idx[:0], wts[:0], w13, w2, workspace=ws)
    assert ep.moe_error(ws) == 0
    for n in (1, 9):                    # nobody names an expert: zeros, whatever was there
        y = torch.full((n, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
        layer(x[:n], torch.full_like(idx[:n], -1), torch.full_like(wts[:n], float("nan")), w13, w2,
              out=y)
        assert torch.equal(y.cpu(), torch.zeros((n, 128), dtype=torch.bfloat16))


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_layer_bad_and_repeated_ids(dtype):
    x, idx, wts, w13, w2 = small()
    idx = idx.to(dtype)
    ws = ep.alloc_moe_workspace(9, 3, 6, 128, 64)
    idx[2] = torch.tensor([4, 4, 4])
    idx[3] = torch.tensor([1, -1, 1])
    want = ref.moe(x, idx, wts, w13, w2)
    held(layer(x, idx, wts, w13, w2, workspace=ws), *want)
    assert ep.moe_error(ws) == 0
    idx[5, 1], idx[6, 0] = 6, -2
    if dtype == torch.int64:
        idx[7, 2] = 2 ** 32 + 1         # no expert, and not expert 1
    want = ref.moe(x, idx, wts, w13, w2)
    held(layer(x, idx, wts, w13, w2, workspace=ws), *want)
    assert ep.moe_error(ws) == ep.EP_LAYOUT_ERR_INDEX
    idx.clamp_(-1, 5)
    layer(x, idx, wts, w13, w2, workspace=ws)
    assert ep.moe_error(ws) == 0


@pytest.mark.parametrize("fmt", ["bf16", "int4", "mxfp4"])
@pytest.mark.parametrize("N", [3, 9, 40])
def test_tokens_do_not_touch_each_other(fmt, N):
    """A token's NaN stays in its row, its neighbours' bits do not change; weights of
    absent choices may be NaN."""
    x, idx, wts, w13, w2 = small(N=N, fmt=fmt)
    idx[1] = torch.tensor([0, 2, 5])
    clean = layer(x, idx, wts, w13, w2).cpu()
    x2, wts2 = x.clone(), wts.clone()
    x2[1] = float("nan")
    wts2[idx < 0] = float("nan")
    y = layer(x2, idx, wts2, w13, w2).cpu()
    assert torch.isnan(y[1]).all()
    keep = torch.arange(N) != 1
    assert torch.equal(y[keep], clean[keep])


def test_layer_repeats_bit_for_bit_and_leaves_inputs_alone():
    for N in (2, 12, 50):
        x, idx, wts, w13, w2 = small(N=N)
        dev = [t.cuda() for t in (x, idx, wts)]
        ws = torch.full((ep.moe_workspace_bytes(N, 3, 6, 128, 64),), 255, dtype=torch.uint8,
                        device="cuda")
        a = ep.moe_layer(*dev, w13.arg, w2.arg, workspace=ws)
        for _ in range(3):
            assert torch.equal(a, ep.moe_layer(*dev, w13.arg, w2.arg))
        for t, d in zip((x, idx, wts), dev):
            assert torch.equal(t, d.cpu())


def test_rows_behind_the_output_stay():
    """Outputs inside larger buffers: what lies before and behind is left alone."""
    x, idx, wts, w13, w2 = small()
    buf = torch.full((11, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    layer(x, idx, wts, w13, w2, out=buf[1:10])
    assert (buf[0] == 3).all() and (buf[10] == 3).all()
    w = ref.W("mxfp4", (), 37, 96, gen=torch.Generator().manual_seed(1))
    buf = torch.full((400,), 3.0, dtype=torch.bfloat16, device="cuda")
    xl = torch.randn((5, 96), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    y = buf[1:1 + 5 * 37].view(5, 37)            # odd rows at an odd offset
    ep.quant_linear(xl.cuda(), w.arg, out=y)
    held(y, *ref.linear(xl, w))
    assert buf[0] == 3 and (buf[1 + 5 * 37:] == 3).all()


def test_route_and_layer_in_graphs_and_streams():
    """Router and layer captured together, two graphs with a workspace each, replayed
    in turn on new inputs with eager work between, against the eager calls."""
    gen = torch.Generator().manual_seed(11)
    _, _, _, w13, w2 = small()
    graphs = []
    for N in (2, 9):
        x = torch.zeros((N, 128), dtype=torch.bfloat16, device="cuda")
        logits = torch.zeros((N, 6), device="cuda")
        out = (torch.empty((N, 3), dtype=torch.int32, device="cuda"),
               torch.empty((N, 3), device="cuda"))
        y, ws = torch.empty_like(x), ep.alloc_moe_workspace(N, 3, 6, 128, 64)
        g = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            ep.route(logits, 3, out=out)
            ep.moe_layer(x, *out, w13.arg, w2.arg, out=y, workspace=ws)
        torch.cuda.current_stream().wait_stream(s)
        with torch.cuda.graph(g):
            ep.route(logits, 3, out=out)
            ep.moe_layer(x, *out, w13.arg, w2.arg, out=y, workspace=ws)
        graphs.append((g, x, logits, y))
    for turn in range(4):
        for g, x, logits, y in graphs:
            x.copy_(torch.randn(x.shape, generator=gen).to(torch.bfloat16))
            logits.copy_(torch.randn(logits.shape, generator=gen))
        for g, *_ in graphs:
            g.replay()
        for g, x, logits, y in graphs:
            want = ep.moe_layer(x, *ep.route(logits, 3), w13.arg, w2.arg)
            torch.cuda.synchronize()
            assert torch.equal(y, want)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()      # two calls at once
    torch.cuda.synchronize()
    got = []
    for s, (g, x, logits, y) in zip((a, b), graphs):
        with torch.cuda.stream(s):
            got.append(ep.moe_layer(x, *ep.route(logits, 3), w13.arg, w2.arg))
    torch.cuda.synchronize()
    for (g, x, logits, y), v in zip(graphs, got):
        assert torch.equal(y, v)


def test_layer_is_dispatch_experts_combine():
    """The layer against the framework's own path: route, layout, dispatch, the
    experts in 64 bits on the dispatched rows, combine."""
    N, H, I, E, K = 24, 256, 128, 8, 2
    gen = torch.Generator().manual_seed(7)
    w13, w2 = ref.W("bf16", (E,), 2 * I, H, gen=gen), ref.W("bf16", (E,), H, I, gen=gen)
    x = torch.randn((N, H), generator=gen).to(torch.bfloat16)
    logits = torch.randn((N, E), generator=gen)
    idx, wts = ep.route(logits.cuda(), K)
    y = ep.moe_layer(x.cuda(), idx, wts, w13.arg, w2.arg)
    lay = ep.get_layout(idx, E, 4)
    recv_x, _, src, _ = ep.dispatch(x.cuda(), wts, lay)
    off, rows = lay.expert_slot_offset.tolist(), recv_x.double().cpu()
    out = torch.zeros_like(rows)
    for e in range(E):
        r = rows[off[e]:off[e + 1]]
        g, u = (r @ w13.value[e].t()).chunk(2, dim=1)
        out[off[e]:off[e + 1]] = (g * torch.sigmoid(g) * u) @ w2.value[e].t()
    out = out.to(torch.bfloat16)
    z = ep.combine(out.cuda(), lay, wts).double().cpu()
    want, bound = ref.moe(x, idx.cpu(), wts.cpu(), w13, w2)
    held(y, want, bound)
    # combine's own roundings: the expert rows and y in bf16, K float32 sums
    rows_mag = torch.zeros_like(want)
    slot = lay.slot_of.cpu()
    for k in range(K):
        rows_mag += wts[:, k].double().cpu()[:, None] * out.double()[slot[:, k].long()].abs()
    assert ((z - y.double().cpu()).abs()
            <= bound + ref.HALF * 1.01 * rows_mag + ref.HALF * z.abs() + 4 * ref.U * rows_mag).all()


@pytest.mark.parametrize("fmt,zeros", [("int4", True), ("mxfp4", False)])
def test_copied_weights_and_rebound_tensors(fmt, zeros):
    """A copy does not read its original, nor a weight what its tensors became since;
    values changed in place count."""
    gen = torch.Generator().manual_seed(12)
    w = ref.W(fmt, (), 40, 256, zeros=zeros, gen=gen)
    x = torch.randn((3, 256), generator=gen).to(torch.bfloat16).cuda()
    want = ep.quant_linear(x, w.arg)
    codes, scales = w.arg.codes.clone(), w.arg.scales.clone()
    v = ep.QuantWeight(codes, scales, zeros=w.arg.zeros, group=w.group, fmt=fmt)
    u = copy.deepcopy(v)
    codes.data, scales.data = torch.zeros_like(codes), torch.zeros_like(scales)
    assert torch.equal(ep.quant_linear(x, v), want)
    v.scales.zero_()                    # 0 of int4, 2^-127 of mxfp4
    tiny = ep.quant_linear(x, v)
    assert (tiny.abs() <= (0 if fmt == "int4" else 2.0 ** -127 * 6 * 256 * 8)).all()
    del v
    assert torch.equal(ep.quant_linear(x, u), want)


@pytest.mark.parametrize("fmt,group,zeros", FORMATS[1:7])
@pytest.mark.parametrize("N", [1, 4, 5, 20])
def test_int4_largest_inputs(fmt, group, zeros, N):
    """|x| up to 2^112: a group's sum of 128 + code, and of its zero point, times x of
    one sign is below 2^112 * 128 * (143 or 255) < 2^127."""
    gen = torch.Generator().manual_seed(N)
    w = ref.W(fmt, (), 40, 256, group, zeros, gen)
    x = (2.0 ** 111 * (1 + torch.rand((N, 256), generator=gen))).to(torch.bfloat16)
    for sign in (1, -1):
        held(ep.quant_linear((sign * x).cuda(), w.arg), *ref.linear(sign * x, w))
