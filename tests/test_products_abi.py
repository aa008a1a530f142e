"""Refusals of the router's and the products' entry points: host checks that
run before any launch, so no GPU is needed."""
import copy
import ctypes
import pickle

import pytest
import torch

import combine_ep_get_amd as ep

FAKE = 256          # never dereferenced: every call here is rejected
FAR = 1 << 30


def route_args(**kw):
    a = ep.RouteArgs(FAKE, None, FAKE, FAKE, 4, 64, 8, 1, 1, 1, 0, 1, 4, 4, 1.0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [
    dict(num_tokens=-1), dict(num_experts=0), dict(num_experts=1025), dict(num_topk=0),
    dict(num_topk=33), dict(num_topk=9, num_groups=8), dict(num_groups=0), dict(num_groups=65),
    dict(num_groups=7), dict(num_groups=8, topk_groups=9), dict(topk_groups=0),
    dict(group_top=0), dict(group_top=3), dict(num_groups=64, topk_groups=64, group_top=2),
    dict(scoring=2), dict(scoring=-1), dict(renormalize=2), dict(logits_bytes=8),
    dict(topk_idx_bytes=2), dict(logits=None), dict(topk_idx=None), dict(topk_weights=None),
    dict(num_tokens=2 ** 31 - 1)], ids=str)
def test_route_refuses(kw):
    assert ep.lib().ep_route(ctypes.byref(route_args(**kw)), None) == 1


def test_null_arguments():
    L = ep.lib()
    assert L.ep_route(None, None) == 1
    p = ep.problem(4, 256, 2, 16, 1)
    assert L.ep_moe_layer(ctypes.byref(p), None, None) == 1
    assert L.ep_moe_layer(None, ctypes.byref(moe_args()), None) == 1
    assert L.ep_moe_workspace_bytes(None, 128) == -1
    assert L.ep_quant_linear(1, 128, 16, FAKE, None, FAKE, None) == 1


def weight(fmt=ep.EP_WEIGHT_BF16, group=0, data=FAKE, scales=FAKE, zeros=None):
    return ep.WeightDesc(data, scales, zeros, fmt, group)


def moe_args(w13=None, w2=None, **kw):
    a = ep.MoeArgs(FAKE, FAKE, FAKE, w13 or weight(), w2 or w13 or weight(), FAKE, FAKE, 128)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def moe_problem(**kw):
    base = dict(num_tokens=4, hidden=256, num_topk=2, num_experts=16, num_ranks=1)
    base.update(kw)
    return ep.problem(**base)


INT4, MX = ep.EP_WEIGHT_INT4, ep.EP_WEIGHT_MXFP4


@pytest.mark.parametrize("pk,ak", [
    (dict(num_tokens=257), {}), (dict(num_tokens=-1), {}), (dict(hidden=0), {}),
    (dict(hidden=12), {}), (dict(hidden=65544), {}), (dict(num_experts=1025), {}),
    (dict(num_topk=33), {}), (dict(topk_idx_bytes=2), {}), ({}, dict(inter=0)),
    ({}, dict(inter=12)), ({}, dict(inter=65544)), ({}, dict(inter=-8)),
    (dict(num_tokens=256, num_topk=32), dict(inter=65536)),
    ({}, dict(x=None)), ({}, dict(topk_idx=None)), ({}, dict(topk_weights=None)),
    ({}, dict(y=None)), ({}, dict(workspace=None)), ({}, dict(workspace=FAKE + 128)),
    ({}, dict(x=FAKE + 2)), ({}, dict(y=FAKE + 1)),
    ({}, dict(w13=weight(data=None))), ({}, dict(w2=weight(data=None))),
    ({}, dict(w13=weight(data=FAKE + 8))), ({}, dict(w13=weight(fmt=3))),
    ({}, dict(w13=weight(INT4, 128), w2=weight(INT4, 64))),
    ({}, dict(w13=weight(INT4, 128), w2=weight(INT4, 128, zeros=FAKE))),
    ({}, dict(w13=weight(INT4, 128), w2=weight())), ({}, dict(w13=weight(INT4, 16))),
    ({}, dict(w13=weight(INT4, 128, scales=None))),
    ({}, dict(w13=weight(INT4, 128, scales=FAKE + 1))),
    ({}, dict(w13=weight(INT4, 128), inter=64)), (dict(hidden=320), dict(w13=weight(INT4, 128))),
    ({}, dict(w13=weight(MX, 64))), ({}, dict(w13=weight(MX, 32, zeros=FAKE))),
    ({}, dict(w13=weight(MX, 32), inter=80))], ids=str)
def test_layer_refuses(pk, ak):
    ak = dict(ak)
    if "w13" in ak and "w2" not in ak:
        ak["w2"] = ak["w13"]
    p = moe_problem(**pk)
    assert ep.lib().ep_moe_layer(ctypes.byref(p), ctypes.byref(moe_args(**ak)), None) == 1


def test_workspace_bytes():
    small = ep.moe_workspace_bytes(1, 8, 32, 7168, 2048)
    assert small >= 8 * 2048 * 2 and small % 256 == 0
    assert ep.moe_workspace_bytes(256, 8, 32, 7168, 2048) >= 256 * 8 * 2048 * 2
    assert ep.moe_workspace_bytes(0, 8, 32, 7168, 2048) > 0
    for K, E, I in ((32, 1024, 8), (1, 3, 8), (8, 32, 2048)):      # for n tokens is for fewer
        sizes = [ep.moe_workspace_bytes(n, K, E, 64, I) for n in range(257)]
        assert sizes == sorted(sizes)
    for bad in ((257, 8, 32, 7168, 2048), (1, 8, 32, 7170, 2048), (1, 8, 32, 7168, 2047),
                (256, 32, 64, 4096, 65536)):
        with pytest.raises(ValueError):
            ep.moe_workspace_bytes(*bad)


@pytest.mark.parametrize("n,cols,rows,w,x,y", [
    (-1, 128, 16, weight(INT4, 128), FAKE, FAR), (257, 128, 16, weight(INT4, 128), FAKE, FAR),
    (1, 0, 16, weight(INT4, 128), FAKE, FAR), (1, 192, 16, weight(INT4, 128), FAKE, FAR),
    (1, 65664, 16, weight(INT4, 128), FAKE, FAR), (1, 128, 0, weight(INT4, 128), FAKE, FAR),
    (1, 128, (1 << 24) + 1, weight(INT4, 128), FAKE, FAR), (1, 128, 16, weight(), FAKE, FAR),
    (1, 128, 16, weight(INT4, 128), None, FAR), (1, 128, 16, weight(INT4, 128), FAKE, None),
    (1, 128, 16, weight(INT4, 128), FAKE + 2, FAR), (1, 48, 16, weight(MX, 32), FAKE, FAR),
    # y over x: the same, its end over x's start, its start over x's end
    (4, 128, 16, weight(INT4, 128), FAKE, FAKE), (4, 128, 16, weight(INT4, 128), FAR, FAR - 126),
    (4, 128, 16, weight(INT4, 128), FAR, FAR + 1022)],
    ids=str)
def test_linear_refuses(n, cols, rows, w, x, y):
    assert ep.lib().ep_quant_linear(n, cols, rows, x, ctypes.byref(w), y, None) == 1


def test_binding_refuses():
    u8, bf16 = torch.uint8, torch.bfloat16
    with pytest.raises(ValueError):                      # not on the GPU
        ep.route(torch.zeros((2, 16)), 4)
    with pytest.raises(ValueError):
        ep.route(torch.zeros((2, 16), dtype=torch.float16), 4)
    with pytest.raises(ValueError):
        ep.QuantWeight(torch.zeros((16, 64), dtype=u8), torch.zeros((16, 1), dtype=bf16))
    with pytest.raises(ValueError):
        ep.QuantWeight(torch.zeros((16, 64), dtype=u8), torch.zeros((16, 1), dtype=bf16), group=16)
    with pytest.raises(ValueError):
        ep.QuantWeight(torch.zeros((16, 64), dtype=u8), torch.zeros((16, 4), dtype=u8), fmt="fp4")
    with pytest.raises(ValueError):
        ep.quant_linear(torch.zeros((2, 128), dtype=bf16), torch.zeros((16, 128), dtype=bf16))
    with pytest.raises(ValueError):
        ep.pack_codes(torch.zeros((4, 12), dtype=u8))
    with pytest.raises(ValueError):
        ep.moe_layer(torch.zeros((2, 64), dtype=bf16), torch.zeros((2, 2), dtype=torch.int32),
                     torch.zeros((2, 2)), torch.zeros((4, 32, 64), dtype=bf16),
                     torch.zeros((4, 64, 16), dtype=bf16))


def test_pack_codes_layout():
    codes = torch.arange(8, dtype=torch.uint8).view(1, 8)
    word = int.from_bytes(bytes(ep.pack_codes(codes)[0].tolist()), "little")
    assert [(word >> 4 * j) & 15 for j in range(8)] == [0, 2, 4, 6, 1, 3, 5, 7]
    assert ep.pack_codes(codes, "mxfp4")[0].tolist() == [0x10, 0x32, 0x54, 0x76]


def test_packed_structs_are_the_structs():
    """The binding packs the C structs into bytes: same sizes, same fields."""
    a = ep.RouteArgs.from_buffer_copy(ep._ROUTE_ARGS(1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14,
                                                     0.5))
    assert [getattr(a, f) for f, _ in a._fields_] == [*range(1, 15), 0.5]
    d = ep.WeightDesc.from_buffer_copy(ep._WEIGHT_DESC(1, 2, 3, 4, 5))
    assert [getattr(d, f) for f, _ in d._fields_] == [1, 2, 3, 4, 5]
    m = ep.MoeArgs.from_buffer_copy(ep._MOE_ARGS(*range(1, 17)))
    flat = [m.x, m.topk_idx, m.topk_weights]
    flat += [getattr(w, f) for w in (m.w13, m.w2) for f, _ in w._fields_]
    assert flat + [m.y, m.workspace, m.inter] == list(range(1, 17))
    p = ep.Problem.from_buffer_copy(ep._PROBLEM(*range(1, 10)))
    assert [getattr(p, f) for f, _ in p._fields_] == list(range(1, 10))
    for packed, struct in ((ep._ROUTE_ARGS(*[0] * 14, 0.0), ep.RouteArgs),
                           (ep._WEIGHT_DESC(*[0] * 5), ep.WeightDesc),
                           (ep._MOE_ARGS(*[0] * 16), ep.MoeArgs),
                           (ep._PROBLEM(*[0] * 9), ep.Problem)):
        assert len(packed) == ctypes.sizeof(struct)


@pytest.mark.parametrize("zeros", [False, True])
def test_quant_weight_is_fixed(monkeypatch, zeros):
    """Calls pass the addresses a weight was made with, so nothing may leave them behind:
    no attribute is rebound, changed storage is noticed, copies have their own."""
    monkeypatch.setattr(ep, "_arg", lambda *a: None)     # CPU tensors will do here
    parts = [torch.zeros((16, 64), dtype=torch.uint8), torch.ones((16, 1), dtype=torch.bfloat16),
             torch.full((16, 1), 8, dtype=torch.uint8) if zeros else None]
    w = ep.QuantWeight(*parts)
    for name in ("codes", "scales", "zeros", "group", "fmt", "shape", "device", "desc", "other"):
        with pytest.raises(AttributeError):
            setattr(w, name, getattr(w, name, None))
        with pytest.raises(AttributeError):
            delattr(w, name)
    desc = w.checked_desc()
    held = [t.clone() for t in parts if t is not None]
    for t in parts:
        if t is not None:
            t.data = torch.zeros(4, dtype=t.dtype)       # the caller's tensor goes elsewhere
    assert w.checked_desc() == desc
    assert all(torch.equal(a, b) for a, b in zip((w.codes, w.scales, w.zeros), held))
    for copied in (copy.deepcopy(w), pickle.loads(pickle.dumps(w))):
        assert copied.desc[0] == copied.codes.data_ptr() != desc[0] and copied.shape == w.shape
        assert copied.desc[3:] == desc[3:] and bool(copied.desc[2]) == zeros
    assert copy.copy(w).checked_desc() == desc           # shares the memory, and holds it
    for t in (w.codes, w.scales, w.zeros):
        if t is not None:
            v = copy.deepcopy(w)
            at = v.codes if t is w.codes else v.scales if t is w.scales else v.zeros
            at.untyped_storage().resize_(0)
            with pytest.raises(ValueError):
                ep._weight_desc(v, v.shape, "w", v)
