"""8-bit products whose scales are at the ends of float32's range."""
import pytest
import torch

import combine_ep_get_amd as ep
from tests import ffn_ref as ref
from tests.test_gpu_ffn import BF, gen, normal

pytestmark = pytest.mark.gpu
ONCE = ref.BF16 + 4 * ref.F32


def weight(g, rows, cols, scale):
    codes = torch.randint(-128, 128, (rows, cols), generator=g, device="cuda").to(torch.int8)
    return ep.Int8Weight(codes, (torch.rand((rows,), generator=g, device="cuda") + 0.5) * scale)


# rows: rounded on the way; few, middle and many
@pytest.mark.parametrize("N,C,O", [(3, 512, 333), (40, 512, 333), (700, 4096, 1022),
                                   (4096, 512, 1024)])
def test_largest_rows_by_smallest_scales(N, C, O):
    """Sums times a row's scale pass float32's largest value, the results do not."""
    g = gen(61)
    x = normal(g, N, C)
    x[0] = (x[0].float() * 1e38).clamp(-3.3e38, 3.3e38).to(BF)
    x[N - 1] = (x[N - 1].float() * 3e36).to(BF)
    w = weight(g, O, C, 1e-36)
    q, s = ref.quantize(x)
    want = (q @ w.codes.double().t()) * s.double()[:, None] * w.scales.double()
    assert float(want.abs().max()) < 1e12
    ref.check(ep.int8_linear(x, w), want, ONCE * want.abs(), "y")
    codes, scales = ep.quantize_int8(x)
    ref.check(ep.int8_linear(codes, w, x_scales=scales), want, ONCE * want.abs(), "y of codes")
    # the other way round, and both at the middle
    scales = scales * 0 + 1e-36
    big = ep.Int8Weight(w.codes, w.scales * 1e36 * 1e30)
    want = (q @ w.codes.double().t()) * scales.double()[:, None] * big.scales.double()
    ref.check(ep.int8_linear(codes, big, x_scales=scales), want, ONCE * want.abs(), "y of tiny rows")


@pytest.mark.parametrize("N,H,I", [(3, 512, 144), (40, 512, 144), (512, 2048, 1024),
                                   (4096, 512, 528)])
def test_largest_rows_of_a_block(N, H, I):
    """gate and up of the largest rows of x are ordinary numbers with such weights."""
    g = gen(62)
    x = normal(g, N, H)
    x[0] = (x[0].float() * 1e38).clamp(-3.3e38, 3.3e38).to(BF)
    w13, w2 = weight(g, 2 * I, H, 1e-42), weight(g, H, I, 1e-3)
    gu = torch.empty((N, 2 * I), dtype=BF, device="cuda")
    y = ep.expert_ffn(x, w13, w2, gate_up=gu)
    q, s = ref.quantize(x)
    want = (q @ w13.codes.double().t()) * s.double()[:, None] * w13.scales.double()
    assert 1e-3 < float(want[0].abs().max()) < 1e6
    ref.check(gu, want, ONCE * want.abs(), "gate_up")
    assert bool(y.isfinite().all())


@pytest.mark.parametrize("off", [1, 2, 3])
@pytest.mark.parametrize("N", [3, 40, 700, 4096])
def test_scales_at_any_float(N, off):
    """Scales that start at any multiple of 4 bytes, of an even and of an odd width."""
    g = gen(63)

    def moved(w):
        s = torch.empty((w.scales.numel() + off,), device="cuda")[off:].view(w.scales.shape)
        assert s.data_ptr() % 16 == 4 * off
        return ep.Int8Weight(w.codes, s.copy_(w.scales))

    for O in (512, 333):
        w, x = weight(g, O, 1024, 1e-2), normal(g, N, 1024)
        assert torch.equal(ep.int8_linear(x, moved(w)), ep.int8_linear(x, w))
    w13, w2 = weight(g, 1056, 1024, 1e-3), weight(g, 1024, 528, 1e-3)
    assert torch.equal(ep.expert_ffn(x, moved(w13), moved(w2)), ep.expert_ffn(x, w13, w2))
    codes, scales = ep.quantize_int8(x)
    s = torch.empty((N + off,), device="cuda")[off:]
    assert torch.equal(ep.int8_linear(codes, w13, x_scales=s.copy_(scales)),
                       ep.int8_linear(codes, w13, x_scales=scales))
