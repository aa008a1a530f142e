"""The router on the GPU against a plain implementation in Python floats: ids equal,
weights within float32's roundings.

Of a weight, with u = 2^-24: exp(x) from a difference of logits x, which is
rounded by u |x|, so that the exponential moves by (|x| + 2) u; the same once more
in a sigmoid's denominator, at most 3 u; its sum u, the quotient 2 u; the sum of
the chosen, K - 1 <= 31 additions in a tree of at most six levels (or a softmax's
sum of up to 1024: 16 in a row, then six levels) of terms with the same errors,
|x| e^-x < 0.4 on the whole: at most 30 u; the quotient and the scale 3 u:
(|x| + 41) u, x the distance from the largest chosen logit (from the row's
maximum where the weights are not divided by their sum; from 0 for a sigmoid)."""
import math

import pytest
import torch

import combine_ep_get_amd as ep
from tests import product_ref as ref

pytestmark = pytest.mark.gpu


def check(logits, K, bias=None, **kw):
    idx, w = ep.route(logits.cuda(), K, bias=None if bias is None else bias.cuda(), **kw)
    kw.pop("idx_dtype", None)
    want_idx, want_w = ref.route(logits, K, bias, **kw)
    assert torch.equal(idx.cpu().long(), want_idx)
    x = torch.nan_to_num(logits.double(), nan=0.0, neginf=0.0).clamp(max=3.402823466e38)
    x = x.gather(1, want_idx.clamp(min=0))
    if kw.get("renormalize", True):
        far = x.amax(dim=1, keepdim=True) - x
    elif kw.get("scoring") == "softmax":
        far = torch.nan_to_num(logits.double(), nan=-math.inf).clamp(max=3.402823466e38) \
            .amax(dim=1, keepdim=True) - x
    else:
        far = x.abs()
    far = torch.where(want_w > 0, far.abs().clamp(max=1e6), torch.zeros_like(far))
    w, want = w.double().cpu(), want_w
    off = (w - want).abs() - (far + 41) * 2.0 ** -24 * want.abs()
    assert (off <= 2.0 ** -125 * kw.get("scale", 1.0)).all(), float(off.max())   # or underflow
    return idx, w


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,E,K,G,keep,top", [
    (1, 256, 8, 8, 4, 2), (70, 256, 8, 1, 1, 1), (9, 1, 1, 1, 1, 1), (33, 64, 6, 8, 3, 1),
    (5, 65, 7, 1, 1, 1), (6, 160, 6, 8, 3, 2), (4, 1024, 32, 64, 7, 2), (13, 100, 10, 4, 4, 1),
    (3, 7, 7, 7, 7, 1), (8, 129, 32, 3, 1, 2)])
def test_route(scoring, with_bias, dtype, N, E, K, G, keep, top):
    gen = torch.Generator().manual_seed(N * E)
    logits = (2 * torch.randn((N, E), generator=gen)).to(dtype)
    bias = 0.2 * torch.randn((E,), generator=gen) if with_bias else None
    check(logits, K, bias, scoring=scoring, num_groups=G, topk_groups=keep, group_top=top,
          renormalize=N % 2 == 0, scale=2.5 if N % 3 else 1.0,
          idx_dtype=torch.int64 if N % 2 else torch.int32)


def test_ties_go_to_the_lowest():
    logits = torch.zeros((3, 300))
    logits[1] = torch.arange(300) % 3
    logits[2, 5:] = -0.0
    check(logits, 32)
    check(logits, 9, num_groups=10, topk_groups=3, group_top=2)
    check(logits, 4, bias=torch.zeros(300), scoring="softmax", num_groups=10, topk_groups=2)


def test_neighbours_that_float32_cannot_tell_apart():
    """Scores that differ by less than a float32 step are ordered as the formula says."""
    gen = torch.Generator().manual_seed(1)
    logits = 8 + 1e-4 * torch.randn((50, 64), generator=gen)
    bias = 1e-3 * torch.randn((64,), generator=gen)
    check(logits, 8, bias)
    check(logits, 8, bias, num_groups=8, topk_groups=4, group_top=2)
    check(20 + torch.randn((50, 64), generator=gen), 8)      # sigmoid is 1 in float32
    check(logits, 8, num_groups=8, topk_groups=4, group_top=2, scoring="softmax")


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masked_and_extreme_logits(scoring, with_bias):
    gen = torch.Generator().manual_seed(2)
    inf, low = math.inf, torch.finfo(torch.float32).min
    logits = torch.randn((9, 40), generator=gen)
    logits[0] = -inf                              # no expert at all
    logits[1] = float("nan")
    logits[2, 3:] = -inf                          # fewer than K
    logits[3, ::2] = float("nan")
    logits[4] = low                               # the lowest number is a number
    logits[5, 1:] = low
    logits[6, 7] = inf
    logits[6, 9] = inf
    logits[7] = -600 + logits[7]                  # scores near the end of float64's range
    logits[8, :39] = -inf
    bias = 0.1 * torch.randn((40,), generator=gen) if with_bias else None
    for kw in (dict(), dict(num_groups=4, topk_groups=2, group_top=1),
               dict(num_groups=4, topk_groups=3, group_top=2), dict(renormalize=False)):
        check(logits, 6, bias, scoring=scoring, **kw)


def test_no_tokens_and_preallocated_outputs():
    idx, w = ep.route(torch.empty((0, 16), device="cuda"), 4)
    assert idx.shape == w.shape == (0, 4)
    logits = torch.randn((5, 16), generator=torch.Generator().manual_seed(3)).cuda()
    out = (torch.full((7, 4), 9, dtype=torch.int64, device="cuda"),
           torch.full((7, 4), 9.0, device="cuda"))
    got = ep.route(logits, 4, out=(out[0][1:6], out[1][1:6]))
    a, b = ep.route(logits, 4)
    assert torch.equal(got[0], a.long()) and torch.equal(got[1], b)
    for t in out:
        assert (t[0] == 9).all() and (t[6] == 9).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_tokens(dtype):
    gen = torch.Generator().manual_seed(4)
    logits = (1.5 * torch.randn((2000, 256), generator=gen)).to(dtype)
    bias = 0.1 * torch.randn((256,), generator=gen)
    check(logits, 8, bias, num_groups=8, topk_groups=4, group_top=2, scale=2.5)
    check(logits, 8, scoring="softmax", renormalize=False)


def test_routes_feed_the_layout():
    logits = torch.randn((64, 32), generator=torch.Generator().manual_seed(5)).cuda()
    logits[3] = -math.inf                          # a token without experts: -1, no slots
    idx, w = ep.route(logits, 4)
    lay = ep.get_layout(idx, 32, 4, 8)
    assert ep.layout_error(lay) == 0
    assert (lay.slot_of[3] == -1).all() and int(lay.num_recv_per_expert.sum()) == 63 * 4


@pytest.mark.parametrize("E,kw", [
    (64, {}), (65, {}), (256, {}), (1024, {}),
    (256, dict(num_groups=8, topk_groups=4, group_top=2)), (300, dict(num_groups=3, topk_groups=2))],
    ids=str)
def test_runs_of_unclear_experts_of_any_length(E, kw):
    """More experts than a wavefront has lanes, none clear of the next in float32."""
    gen = torch.Generator().manual_seed(E)
    noise = torch.randn((6, E), generator=gen)
    flat = lambda v: torch.full((E,), v)                            # noqa: E731
    check(20 + noise, 8, flat(0.0), **kw)             # every float32 score is 1
    check(-22 + noise, 8, flat(0.1), **kw)
    check(8 + 1e-4 * noise, 8, flat(0.1), **kw)
    check(noise, 8, flat(1e6), **kw)
    for above, b in ((25.0, 0.1), (110.0, 0.0)):      # the rest's scores vanish in float32
        logits = noise.clone()
        logits[torch.arange(6), torch.randint(0, E, (6,), generator=gen)] += above
        check(logits, 8, flat(b), scoring="softmax", **kw)
    if not kw:                                        # clear groups of unclear experts
        for G in (g for g in (1, 2, 3) if E % g == 0):
            by_group = torch.arange(G).repeat_interleave(E // G).float()
            check(20 + noise, 8, by_group, num_groups=G, topk_groups=1, group_top=2)



@pytest.mark.parametrize("E,G", [(32, 4), (48, 4), (256, 8), (1024, 64)])
def test_group_scores_of_large_opposite_terms(E, G):
    """Biases that cancel inside a group: the sum is small, what its terms lost is not."""
    gen = torch.Generator().manual_seed(E)
    a = 0.2 + 0.5 * torch.rand((40, G), generator=gen, dtype=torch.float64)
    b = 0.93 - a + 1e-6 * torch.randn((40, G), generator=gen, dtype=torch.float64)
    logits = torch.zeros((40, G, E // G))
    logits[:, :, 1], logits[:, :, 3] = torch.logit(a).float(), torch.logit(b).float()
    for big in (100.0, 1e4):
        bias = torch.full((G, E // G), -1e5)
        bias[:, 1], bias[:, 3] = big, -big
        check(logits.view(40, E), 2, bias.view(-1), num_groups=G, topk_groups=G // 2, group_top=2)



@pytest.mark.parametrize("E,G", [(16, 2), (12, 2), (256, 2)])
def test_group_scores_below_the_lowest_float32(E, G):
    """A group whose two terms add up to less than the lowest float32 still comes
    before one that has too few experts."""
    logits = torch.randn((3, E), generator=torch.Generator().manual_seed(6))
    logits[:, 1:E // 2] = -math.inf
    check(logits, 2, torch.full((E,), -3e38), num_groups=G, topk_groups=1, group_top=2)



def test_a_bias_of_zero_changes_nothing():
    """Divided by their sum the weights do not depend on the row's other scores."""
    logits = torch.randn((500, 200), generator=torch.Generator().manual_seed(8)).cuda()
    a = ep.route(logits, 6, scoring="softmax")
    b = ep.route(logits, 6, scoring="softmax", bias=torch.zeros(200, device="cuda"))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])



@pytest.mark.parametrize("N", [2 ** 26 + 3, 2 ** 31 - 1])
def test_most_tokens(N):
    """More tokens than one grid has wavefronts for, up to the most that are accepted."""
    logits = torch.empty((N, 2), dtype=torch.bfloat16, device="cuda")
    for a in range(0, N, 2 ** 26):
        logits[a:a + 2 ** 26].normal_()
    idx, w = ep.route(logits, 1, scale=1.5)
    for a in range(0, N, 2 ** 26):
        part = logits[a:a + 2 ** 26]
        assert torch.equal(idx[a:a + 2 ** 26, 0], (part[:, 1] > part[:, 0]).int())
        assert (w[a:a + 2 ** 26] == 1.5).all()
