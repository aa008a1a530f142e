"""What the experts' block, its gradient, combine's gradient and the 8-bit products
refuse, on the host: no device is touched (device pointers here are made up)."""
import copy
import ctypes
import pickle

import pytest
import torch

import combine_ep_get_amd as ep
from tests import ffn_ref as ref

INVALID = 1
A, B, C, D, E_, F, G, H_, W = (i << 32 for i in range(1, 10))     # far apart, aligned
BF16, INT4, INT8 = ep.EP_WEIGHT_BF16, ep.EP_WEIGHT_INT4, ep.EP_WEIGHT_INT8


def rows(offset=A, count=A + 4096, capacity=64, num_experts=4, num_sources=1, rows_per_source=0,
         max_rows=32):
    return ep.RowsDesc(offset, count, capacity, num_experts, num_sources, rows_per_source, max_rows)


def plain(n=8, cap=8):
    return rows(None, None, cap, 1, 1, 0, n)


def blocks(**kw):
    return rows(**{**dict(offset=None, capacity=64, num_experts=4, num_sources=2,
                          rows_per_source=8), **kw})


def weight(fmt=BF16, data=D, scales=None):
    return ep.WeightDesc(data, scales, None, fmt, 0)


def accepted(rc):
    """Past every check: without a device the next is the device itself."""
    return rc in ((0, 3, 4) if torch.cuda.is_available() else (3, 4))


BAD_ROWS = [
    None, rows(capacity=-1), rows(capacity=1 << 31), rows(max_rows=-1), rows(num_experts=0),
    rows(num_experts=1025), rows(num_sources=0), rows(num_sources=257), rows(count=None),
    rows(num_sources=2), rows(rows_per_source=1), rows(offset=A + 2), rows(count=A + 1),
    blocks(rows_per_source=0), blocks(rows_per_source=9), blocks(rows_per_source=-1),
    rows(None, None, 64, 4), rows(None, None, 8, 1, 1, 0, 9), rows(None, None, 8, 1, 2, 0, 8),
    rows(None, None, 8, 1, 1, 4, 8)]


def ffn(r, x=B, w13=None, w2=None, y=C, gate_up=None, workspace=W, hidden=64, inter=32):
    a = ep.FfnArgs(x, w13 or weight(), w2 or weight(data=E_), y, gate_up, workspace, hidden, inter)
    return ep.lib().ep_ffn(None if r is None else ctypes.byref(r), ctypes.byref(a), None)


def grad(r, **kw):
    d = dict(dy=A, x=B, gate_up=C, w13=D, w2=E_, dx=F, dw13=G, dw2=H_, workspace=W, hidden=64,
             inter=32)
    a = ep.FfnGradArgs(*{**d, **kw}.values())
    return ep.lib().ep_ffn_backward(None if r is None else ctypes.byref(r), ctypes.byref(a), None)


def integer(r, x=B, x_scales=None, w=None, y=C, workspace=W, cols=64, out_rows=40):
    a = ep.Int8Args(x, x_scales, w or weight(INT8, scales=E_), y, workspace, cols, out_rows)
    return ep.lib().ep_integer_linear(None if r is None else ctypes.byref(r), ctypes.byref(a), None)


@pytest.mark.parametrize("i", range(len(BAD_ROWS)))
def test_rows_refused(i):
    r = BAD_ROWS[i]
    assert ffn(r) == INVALID and grad(r) == INVALID and integer(r) == INVALID
    ptr = None if r is None else ctypes.byref(r)
    assert ep.lib().ep_ffn_workspace_bytes(ptr, 64, 32, BF16, 0) == -1
    assert ep.lib().ep_integer_workspace_bytes(ptr, 64) == -1


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers: host only")


@no_gpu
def test_good_arguments_reach_the_device_check():
    for r in (rows(), plain(), blocks()):
        assert accepted(ffn(r)) and accepted(integer(r))
        assert accepted(ffn(r, y=B)) and accepted(ffn(r, gate_up=F))
        assert accepted(integer(r, x_scales=F, workspace=None))
    assert accepted(grad(rows())) and accepted(grad(plain()))
    assert accepted(grad(rows(max_rows=0), dy=None, x=None, gate_up=None, dx=None, workspace=None))


def test_no_rows_do_nothing():
    assert ffn(rows(max_rows=0), x=None, y=None) == 0
    assert integer(plain(0, 0), x=None, y=None) == 0
    assert ep.lib().ep_quantize_rows(0, 16, None, None, None, None) == 0


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(y=None), dict(workspace=None), dict(w13=weight(data=None)),
    dict(w2=weight(data=None)), dict(x=B + 8), dict(y=C + 2), dict(workspace=W + 128),
    dict(gate_up=F + 8), dict(w13=weight(data=D + 8)), dict(w2=weight(INT8, scales=F)),
    dict(w13=weight(INT4), w2=weight(INT4)), dict(w13=weight(INT8), w2=weight(INT8)),
    dict(w13=weight(INT8, scales=F + 2), w2=weight(INT8, scales=G)),
    dict(hidden=0), dict(hidden=60), dict(hidden=65544), dict(inter=0), dict(inter=-8),
    dict(inter=36), dict(inter=65544),
    dict(w13=weight(INT8, scales=F), w2=weight(INT8, scales=G), hidden=72),
    dict(w13=weight(INT8, scales=F), w2=weight(INT8, scales=G), inter=40),
    dict(gate_up=B), dict(gate_up=C), dict(gate_up=C + 64 * 128 - 16)], ids=str)
def test_ffn_refuses(kw):
    assert ffn(rows(), **kw) == INVALID


@pytest.mark.parametrize("kw", [
    *[{n: None} for n in ("dy", "x", "gate_up", "w13", "w2", "dx", "dw13", "dw2", "workspace")],
    *[{n: 3 * (1 << 40) + 8} for n in ("dy", "x", "gate_up", "w13", "w2", "dx", "dw13", "dw2",
                                       "workspace")],
    dict(hidden=0), dict(hidden=12), dict(inter=65544),
    # an output over an input: the same, its start, its end
    dict(dx=A), dict(dx=B), dict(dx=C), dict(dx=B + 64 * 128 - 16), dict(dx=B - 64 * 128 + 16),
    dict(dw13=D), dict(dw2=E_), dict(dw2=A), dict(dw13=C)], ids=str)
def test_backward_refuses(kw):
    assert grad(rows(), **kw) == INVALID


def test_backward_refuses_sub_blocks():
    assert grad(blocks()) == INVALID


@no_gpu
def test_tiles_of_overlapping_regions_fit():
    assert accepted(ffn(rows(capacity=1 << 20, num_experts=1024)))


def test_tiles_beyond_32_bits():
    """Counts that give every expert the whole buffer must leave the tiles countable."""
    big = rows(capacity=1 << 27, num_experts=1024)
    assert ffn(big) == INVALID and integer(big, y=1 << 46) == INVALID


def test_sub_blocks_beyond_32_bits():
    """Offsets inside an expert's sub-blocks have 32 bits: larger ones are refused."""
    big = blocks(capacity=1 << 30, num_experts=1, num_sources=64, rows_per_source=1 << 16)
    assert ffn(big, hidden=7168, inter=2048) == INVALID and integer(big, cols=7168) == INVALID


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(y=None), dict(workspace=None), dict(x=B + 4), dict(y=C + 2),
    dict(workspace=W + 64), dict(w=weight(INT8)), dict(w=weight(BF16, scales=E_)),
    dict(w=weight(INT8, data=None, scales=E_)), dict(w=weight(INT8, data=D + 8, scales=E_)),
    dict(w=weight(INT8, scales=E_ + 2)), dict(x_scales=F + 2), dict(cols=0), dict(cols=24),
    dict(cols=65552), dict(out_rows=0), dict(out_rows=(1 << 24) + 1), dict(y=B),
    dict(y=B + 64 * 128 - 16), dict(x_scales=F, y=B + 64 * 64 - 16)], ids=str)
def test_integer_linear_refuses(kw):
    assert integer(rows(), **kw) == INVALID


@pytest.mark.parametrize("n,cols,x,codes,scales", [
    (-1, 16, A, B, C), (1 << 31, 16, A, B, C), (1, 0, A, B, C), (1, 8, A, B, C),
    (1, 65552, A, B, C), (1, 16, None, B, C), (1, 16, A, None, C), (1, 16, A, B, None),
    (1, 16, A + 8, B, C), (1, 16, A, B + 8, C), (1, 16, A, B, C + 2), (1, 16, A, A + 16, C),
    (4, 16, A, A - 48, C)])
def test_quantize_refuses(n, cols, x, codes, scales):
    assert ep.lib().ep_quantize_rows(n, cols, x, codes, scales, None) == INVALID


@pytest.mark.parametrize("kw", [
    dict(p=dict(hidden=0)), dict(p=dict(hidden=12)), dict(p=dict(num_tokens=-1)),
    dict(p=dict(num_topk=33)), dict(cap=-1), dict(cap=1 << 31), dict(dy=None), dict(slot=None),
    dict(wts=None), dict(dwts=None), dict(eo=None), dict(deo=None), dict(dy=A + 8),
    dict(eo=B + 8), dict(deo=C + 8), dict(deo=A), dict(deo=B + 16), dict(deo=A + 4 * 128 - 16)],
    ids=str)
def test_combine_backward_refuses(kw):
    d = dict(num_tokens=4, hidden=64, num_topk=2, num_experts=4, num_ranks=1)
    p = ep.problem(**{**d, **kw.get("p", {})})
    g = {**dict(dy=A, eo=B, slot=D, wts=E_, deo=C, dwts=F, cap=8), **kw}
    assert ep.lib().ep_combine_backward(ctypes.byref(p), g["dy"], g["eo"], g["slot"], g["wts"],
                                        g["deo"], g["dwts"], g["cap"], None) == INVALID


def test_workspace_bytes():
    assert ep.ffn_workspace_bytes(0, 64, 32) == 0
    for n in (1, 1000):
        fwd, back, int8 = (ep.ffn_workspace_bytes(n, 256, 128, **kw)
                           for kw in ({}, dict(backward=True), dict(int8=True)))
        assert fwd >= n * 128 * 2 and back >= n * 128 * 6 and int8 >= n * (256 + 3 * 128 + 8)
        assert fwd % 256 == back % 256 == int8 % 256 == 0
    assert ep.ep_integer_workspace_bytes(10, 64) >= 10 * 68
    for bad in (dict(hidden=12), dict(inter=0), dict(rows=-1), dict(int8=True, inter=24),
                dict(int8=True, backward=True)):
        with pytest.raises(ValueError):
            ep.ffn_workspace_bytes(**{**dict(rows=4, hidden=64, inter=32), **bad})
    with pytest.raises(ValueError):
        ep.ep_integer_workspace_bytes(4, 24)


def test_binding_refuses(monkeypatch):
    bf = torch.bfloat16
    x, w13, w2 = torch.zeros((4, 64), dtype=bf), torch.zeros((64, 64), dtype=bf), \
        torch.zeros((64, 32), dtype=bf)
    with pytest.raises(ValueError, match="on the GPU"):
        ep.expert_ffn(x, w13, w2)
    with pytest.raises(ValueError, match="on the GPU"):
        ep.combine_backward(x, x, ep.LLLayout(4, 1, 1, 1, 4, 4, None, x, None), x)
    with pytest.raises(ValueError, match="on the GPU"):
        ep.quantize_int8(x)
    with pytest.raises(ValueError, match="Int8Weight"):
        ep.int8_linear(x, w13)

    def shapes_alone(t, dtype, shape, name, ref):        # CPU tensors will do from here on
        if tuple(t.shape) != tuple(shape):
            raise ValueError(name)
    monkeypatch.setattr(ep, "_arg", shapes_alone)
    q = ep.Int8Weight(torch.zeros((64, 64), dtype=torch.int8), torch.zeros(64))
    q2 = ep.Int8Weight(torch.zeros((64, 32), dtype=torch.int8), torch.zeros(64))
    ll = ep.LLLayout(4, 2, 2, 1, 4, 8, torch.zeros((2, 1)), None, None)
    q3 = ep.Int8Weight(torch.zeros((3, 64, 64), dtype=torch.int8), torch.zeros((3, 64)))
    four = ep.QuantWeight(torch.zeros((64, 32), dtype=torch.uint8), torch.zeros((64, 1), dtype=bf),
                          group=64)
    stack = torch.zeros((3, 64, 64), dtype=bf), torch.zeros((3, 64, 32), dtype=bf)
    for call in (lambda: ep.expert_ffn(x, w13, q2), lambda: ep.expert_ffn(x, q, w2),
                 lambda: ep.expert_ffn(x, w13[:62], w2), lambda: ep.expert_ffn(x, w13, w2[:32]),
                 lambda: ep.expert_ffn(x, *stack),                       # no layout
                 lambda: ep.expert_ffn(x, stack[0], stack[1][:2]),
                 lambda: ep.expert_ffn(x, *stack, layout=ll),            # three of two experts
                 lambda: ep.expert_ffn(x, stack[0][:2], stack[1][:2], layout=ll),   # 4 of 8 rows
                 lambda: ep.expert_ffn(x, w13, w2, workspace=torch.zeros(8, dtype=torch.uint8)),
                 lambda: ep.expert_ffn_backward(x, x, x, q, q2),
                 lambda: ep.expert_ffn_backward(x, x, x, w13, w2, layout=ll),
                 lambda: ep.expert_ffn(x, w13, four), lambda: ep.expert_ffn(x, four, w2),
                 lambda: ep.expert_ffn_backward(x, x, x, w13, four),
                 lambda: ep.moe_layer(x, x[:, :2].int(), x[:, :2], q3, q3),
                 lambda: ep.int8_linear(x[:, :32], q), lambda: ep.int8_linear(x, q, layout=ll),
                 lambda: ep.Int8Weight(torch.zeros((4, 24), dtype=torch.int8), torch.zeros(4)),
                 lambda: ep.Int8Weight(torch.zeros(16, dtype=torch.int8), torch.zeros(1))):
        with pytest.raises(ValueError):
            call()


def test_int8_weight_is_fixed(monkeypatch):
    monkeypatch.setattr(ep, "_arg", lambda *a: None)
    parts = torch.ones((8, 16), dtype=torch.int8), torch.ones(8)
    w = ep.Int8Weight(*parts)
    for name in ("codes", "scales", "shape", "desc", "device", "other"):
        with pytest.raises(AttributeError):
            setattr(w, name, None)
        with pytest.raises(AttributeError):
            delattr(w, name)
    desc = w.checked_desc()
    parts[0].data = torch.zeros(4, dtype=torch.int8)     # the caller's tensor goes elsewhere
    assert w.checked_desc() == desc and bool((w.codes == 1).all())
    for c in (copy.deepcopy(w), pickle.loads(pickle.dumps(w))):
        assert c.desc[0] == c.codes.data_ptr() != desc[0] and c.shape == w.shape
        c.codes.untyped_storage().resize_(0)
        with pytest.raises(ValueError):
            c.checked_desc()


def test_packed_structs_are_the_structs():
    r = ep.RowsDesc.from_buffer_copy(ep._ROWS(*range(1, 8)))
    assert [getattr(r, f) for f, _ in r._fields_] == list(range(1, 8))
    a = ep.FfnArgs.from_buffer_copy(ep._FFN_ARGS(*range(1, 17)))
    flat = [a.x] + [getattr(w, f) for w in (a.w13, a.w2) for f, _ in w._fields_]
    assert flat + [a.y, a.gate_up, a.workspace, a.hidden, a.inter] == list(range(1, 17))
    g = ep.FfnGradArgs.from_buffer_copy(ep._FFN_GRAD_ARGS(*range(1, 12)))
    assert [getattr(g, f) for f, _ in g._fields_] == list(range(1, 12))
    q = ep.Int8Args.from_buffer_copy(ep._INT8_ARGS(*range(1, 12)))
    flat = [q.x, q.x_scales] + [getattr(q.w, f) for f, _ in q.w._fields_]
    assert flat + [q.y, q.workspace, q.cols, q.out_rows] == list(range(1, 12))


# ------------------------------------------------------------------ the oracle itself
def test_reference_gradients_are_those_of_differences():
    """The formulas the GPU is held to against central differences in 64 bits."""
    g = torch.Generator().manual_seed(0)
    n, H, I = 3, 5, 4
    x, w13, w2, dy = (torch.randn(s, generator=g, dtype=torch.float64)
                      for s in ((n, H), (2 * I, H), (H, I), (n, H)))
    grads = [v[0] for v in ref.ffn_grad(dy, x, x @ w13.t(), w13, w2)]
    for t, want in zip((x, w13, w2), grads):
        got = torch.zeros_like(t)
        for i in range(t.numel()):
            v = t.view(-1)[i].item()
            side = []
            for d in (1e-5, -1e-5):
                t.view(-1)[i] = v + d
                side.append((ref.ffn(x, w13, w2)[0] * dy).sum())
            t.view(-1)[i] = v
            got.view(-1)[i] = (side[0] - side[1]) / 2e-5
        assert torch.allclose(got, want, rtol=0, atol=1e-7)


def test_reference_codes():
    """Halves go to even, zeros get scale 1, the extremes are +-127."""
    x = torch.tensor([[127.0, 0.5, 1.5, -0.5, -2.5, -127.0], [0.0] * 6]).to(torch.bfloat16)
    q, s = ref.quantize(x)
    assert q.tolist() == [[127, 0, 2, 0, -2, -127], [0] * 6] and s.tolist() == [1.0, 1.0]
