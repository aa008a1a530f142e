"""The check of the block with 8-bit weights on itself: what float32 makes of it passes, small
faults do not (on the CPU)."""
import pytest
import torch

from tests import ffn_ref as ref
from tests import ffn_tight as tight

BF = torch.bfloat16


def float32_block(x, w13, w2):
    """The block as float32 computes it, with codes and sums as whole numbers."""
    def product(rows, q, s):
        codes, scale = ref.quantize(rows)
        sums = (codes @ q.double().t()).float()            # exact below 2^24, else rounded
        return sums * scale[:, None] * s
    both = product(x, *w13)
    I = both.shape[1] // 2
    a, b = both[:, :I], both[:, I:]
    h = a * (1 / (1 + torch.exp(-a))) * b
    return both.to(BF), product(h.to(BF), *w2).to(BF)


def case(N, H, I, seed=71):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((N, H), generator=g).to(BF)
    w = [ref.quantize((torch.randn(s, generator=g) * s[1] ** -0.5).to(BF))
         for s in ((2 * I, H), (H, I))]
    return (x, *[(q.to(torch.int8), s) for q, s in w])


SIZES = [(300, 272, 208), (96, 1008, 528), (40, 4080, 2064)]


@pytest.mark.parametrize("N,H,I", SIZES)
def test_float32_passes(N, H, I):
    x, w13, w2 = case(N, H, I)
    gu, y = float32_block(x, w13, w2)
    want, choices = tight.block(x, w13, w2)
    tight.check_gate_up(gu, want, "gate_up")
    tight.check_rows(y, choices, "y")
    # and the bound is not much wider than the rounding of y: a tenth of the values' size
    for v, bound in choices:
        assert float((bound - tight.ONCE * v.abs()).max()) < 0.1 * float(v.pow(2).mean().sqrt())


@pytest.mark.parametrize("N,H,I", SIZES)
def test_small_faults_do_not_pass(N, H, I):
    x, w13, w2 = case(N, H, I)
    _, y = float32_block(x, w13, w2)
    _, choices = tight.block(x, w13, w2)

    def refuses(change):
        t = y.clone()
        change(t)
        with pytest.raises(AssertionError):
            tight.check_rows(t, choices, "y")

    def zero(r, c):
        def change(t):
            t[r, c] = 0
        return change
    for r in (0, N // 2, N - 1):
        for c in (0, H // 2 // 8 * 8, H - 8):
            refuses(zero(r, slice(c, c + 8)))              # one chunk of one row
    refuses(zero(slice(None), H - 1))                      # one column

    def neighbour(t):                                      # a column with the next one's scale
        t[:, 5] = (t[:, 5].float() * (w2[1][6] / w2[1][5])).to(BF)
    if abs(float(w2[1][6] / w2[1][5]) - 1) > 0.02:
        refuses(neighbour)

    def shifted(t):                                        # the last row is that before it
        t[-1] = t[-2]
    refuses(shifted)


def test_a_lost_part_of_the_contraction_does_not_pass():
    """The last 16 of 208 values of h left out of the second product."""
    x, w13, w2 = case(300, 272, 208)
    _, choices = tight.block(x, w13, w2)
    q = w2[0].clone()
    q[:, -16:] = 0
    with pytest.raises(AssertionError):
        tight.check_rows(float32_block(x, w13, (q, w2[1]))[1], choices, "y")
