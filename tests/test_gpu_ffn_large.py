"""More tokens than one grid has threads for, and as many rows as 32 bits count."""
import pytest
import torch

import combine_ep_get_amd as ep

pytestmark = pytest.mark.gpu


def test_combine_backward_many_tokens():
    """2^26 tokens and some more: at 64 threads each, more than the 2^32 - 1 threads of a grid."""
    N, H = (1 << 26) + 5, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(41)
    dy = torch.randn((N, H), generator=g, device="cuda", dtype=torch.bfloat16)
    eo = torch.randn((N, H), generator=g, device="cuda", dtype=torch.bfloat16)
    wts = torch.rand((N, 1), generator=g, device="cuda")
    slot = torch.arange(N - 1, -1, -1, dtype=torch.int32, device="cuda").view(N, 1)
    slot[12345] = -1
    lay = ep.LLLayout(N, 1, 1, 1, N, N, None, slot, None)
    deo = torch.full((N, H), 7.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((N, 1), float("nan"), device="cuda")
    ep.combine_backward(dy, eo, lay, wts, out=(deo, dw))
    # one product in float32, rounded to bf16: the same bits whoever computes it
    bits = lambda t: t.view(torch.int16)                                  # noqa: E731
    at = slot[:, 0].long()
    for a in range(0, N, 1 << 24):
        t = torch.arange(a, min(a + (1 << 24), N), device="cuda")
        t = t[at[t] >= 0]
        want = (wts[t] * dy[t].float()).to(torch.bfloat16)
        assert torch.equal(bits(deo[at[t]]), bits(want))
        o = eo[at[t]].double() * dy[t].double()
        err = (dw[t, 0].double() - o.sum(dim=1)).abs()
        assert bool((err <= H * 2.0 ** -24 * o.abs().sum(dim=1)).all())
    assert bool((deo[N - 1 - 12345] == 7.0).all()) and float(dw[12345]) == 0.0


def test_most_rows():
    """2^31 - 1 rows: one more tile of them than whole ones, counted in 32 bits."""
    N, C, O = 2 ** 31 - 1, 16, 1
    g = torch.Generator(device="cuda")
    g.manual_seed(42)
    x = torch.zeros((N, C), dtype=torch.int8, device="cuda")
    ends = [slice(0, 70), slice(1 << 30, (1 << 30) + 70), slice(N - 200, N)]
    for s in ends:
        x[s] = torch.randint(-128, 128, x[s].shape, generator=g, device="cuda").to(torch.int8)
    w = ep.Int8Weight(torch.randint(-128, 128, (O, C), generator=g, device="cuda").to(torch.int8),
                      torch.full((O,), 0.5, device="cuda"))
    y = torch.full((N, O), float("nan"), dtype=torch.bfloat16, device="cuda")
    ep.int8_linear(x, w, x_scales=torch.ones((N,), device="cuda"), out=y)
    for s in ends:
        want = 0.5 * (x[s].double() @ w.codes.double().t())     # exact in float32 too
        assert torch.equal(y[s], want.float().to(torch.bfloat16))
        y[s] = 0
    for a in range(0, N, 1 << 28):
        assert not bool(y[a:a + (1 << 28)].any()), f"rows from {a} on"
