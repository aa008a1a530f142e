"""dispatch and combine of more (token, piece) items than the threads of one grid allow."""
import pytest
import torch

import combine_ep_get_amd as ep

pytestmark = pytest.mark.gpu
STEP = 1 << 24


def layout(N):
    """One expert that has every other token: tokens 1, 3, ... have no slot."""
    idx = torch.zeros((N, 1), dtype=torch.int32, device="cuda")
    idx[1::2] = -1
    lay = ep.get_layout(idx, 1, 1)
    assert int(lay.num_recv_per_expert) == (N + 1) // 2
    assert torch.equal(lay.slot_of[::2, 0], torch.arange((N + 1) // 2, dtype=torch.int32, device="cuda"))
    return lay


def noise(N, H, dtype, seed):
    """Random bits of finite values."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = torch.empty((N, H), dtype=dtype, device="cuda")
    for a in range(0, N, STEP):
        t[a:a + STEP] = torch.randn(t[a:a + STEP].shape, generator=g, device="cuda",
                                    dtype=torch.bfloat16).to(dtype)
    return t


def same(a, b):
    """a[i] == b[2 i], bit by bit."""
    for i in range(0, len(a), STEP):
        x = a[i:i + STEP].view(torch.uint8)
        assert torch.equal(x, b[2 * i:2 * (i + len(x)):2].view(torch.uint8)), f"rows from {i} on"


def check_tags(rw, src, wts, n):
    """The used slots carry their token and weight, the rest of the buffer is marked unused."""
    for i in range(0, n, STEP):
        j = torch.arange(i, min(i + STEP, n), device="cuda")
        assert torch.equal(src[j].long(), 2 * j) and torch.equal(rw[j], wts[2 * j, 0])
    assert bool((src[n:] == -1).all()) and bool((rw[n:] == 0).all())


def test_bf16_and_combine():
    """2^26 and some more: dispatch's workgroups have 256 threads, combine's 64."""
    N, H = (1 << 26) + 5, 8
    lay, x = layout(N), noise(N, H, torch.bfloat16, 1)
    wts = torch.rand((N, 1), device="cuda")
    rx, _, src, rw = ep.dispatch(x, wts, lay)
    n = (N + 1) // 2
    same(rx[:n], x)
    check_tags(rw, src, wts, n)
    y = ep.combine(rx, lay, torch.ones_like(wts), out=torch.full_like(x, 7.0))
    same(rx[:n], y)
    for i in range(0, N // 2, STEP):
        assert not bool(y[1 + 2 * i:1 + 2 * (i + STEP):2].any())


@pytest.mark.parametrize("given", [False, True], ids=["bf16", "codes"])
def test_e4m3(given):
    N, H = (1 << 26) + 5, 128
    lay = layout(N)
    n = (N + 1) // 2
    out = ep.alloc_recv(lay, H, True, "cuda")
    wts = torch.rand((N, 1), device="cuda")
    if given:
        x = noise(N, H, torch.float8_e4m3fn, 2)
        xs = torch.rand((N, 1), device="cuda")
        rx, rs, src, rw = ep.dispatch(x, wts, lay, use_fp8=True, x_scales=xs, out=out)
        same(rx[:n], x)
        same(rs[:n], xs)
    else:
        x = noise(N, H, torch.bfloat16, 3)
        rx, rs, src, rw = ep.dispatch(x, wts, lay, use_fp8=True, out=out)
        for i in range(0, n, STEP):        # a code is off by at most half a step, or a subnormal's
            v, s = x[2 * i:2 * (i + STEP):2][:n - i].float(), rs[i:i + STEP]
            got = rx[i:i + STEP][:len(v)].float() * s[:len(v)]
            assert bool(((got - v).abs() <= 2 ** -4 * v.abs() + 2 ** -10 * s[:len(v)] + 1e-6).all())
    check_tags(rw, src, wts, n)
