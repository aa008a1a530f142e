"""The expert layer at sizes of real models, where it takes other ways than at
small ones: scales 16 bytes of a row at a time in the second product, pairs of row
tiles, contractions of many steps shared out between wavefronts, x shared between
wavefronts in whole steps.  Against the plain 64-bit implementation."""
import functools

import pytest
import torch

import combine_ep_get_amd as ep
from tests import product_ref as ref
from tests.test_gpu_products import held

pytestmark = pytest.mark.gpu

QUANT = [("int4", 128, False), ("int4", 128, True), ("int4", 64, False), ("int4", 64, True),
         ("int4", 32, False), ("int4", 32, True), ("mxfp4", 32, False)]


@functools.lru_cache(maxsize=1)
def weights(fmt, group, zeros, E, H, I):
    gen = torch.Generator().manual_seed(H + I)
    return ref.W(fmt, (E,), 2 * I, H, group, zeros, gen), ref.W(fmt, (E,), H, I, group, zeros, gen)


def check(w13, w2, N, K, absent=0.1, spoil=lambda idx: None):
    gen = torch.Generator().manual_seed(N)
    E, H, _ = w2.value.shape
    x = torch.randn((N, H), generator=gen).to(torch.bfloat16)
    idx = torch.randint(0, E, (N, K), generator=gen, dtype=torch.int32)
    idx[torch.rand((N, K), generator=gen) < absent] = -1
    spoil(idx)
    wts = torch.rand((N, K), generator=gen) + 0.1
    y = ep.moe_layer(x.cuda(), idx.cuda(), wts.cuda(), w13.arg, w2.arg)
    held(y, *ref.moe_by_expert(x, idx, wts, w13, w2, "cuda"))


# 2 tokens to each of 3 experts at most, then lists of about 9, 27 (two items, or
# three of 16 tokens), 47 and 130 tokens
@pytest.mark.parametrize("N", [3, 13, 40, 70, 200])
@pytest.mark.parametrize("fmt,group,zeros,I", [(*f, 1024) for f in QUANT]
                         + [("int4", 128, False, 2048), ("mxfp4", 32, False, 2048),
                            ("int4", 128, True, 1152), ("mxfp4", 32, False, 1056),
                            ("bf16", None, False, 1400)])
def test_second_product(fmt, group, zeros, I, N):
    check(*weights(fmt, group, zeros, 3, 6144 + 128, I), N, 2)


@pytest.mark.parametrize("N", [2, 4, 5, 16, 33])
@pytest.mark.parametrize("fmt,group,zeros", QUANT + [("bf16", None, False)])
def test_second_product_of_one_expert(fmt, group, zeros, N):
    """All tokens to one of two experts: few items, each of them split over wavefronts."""
    def spoil(idx):
        idx[:] = 1
    check(*weights(fmt, group, zeros, 2, 1024, 2048), N, 1, spoil=spoil)


@pytest.mark.parametrize("N", [33, 60])
@pytest.mark.parametrize("fmt,group,zeros,E,H,I", [
    ("int4", 128, False, 260, 1024, 128), ("int4", 128, True, 260, 1024, 128),
    ("int4", 64, False, 130, 1024, 128), ("int4", 64, True, 130, 512, 128),
    ("int4", 32, False, 130, 768, 128), ("int4", 32, True, 130, 768, 128),
    ("mxfp4", 32, False, 260, 512, 128)])
def test_shared_x(fmt, group, zeros, E, H, I, N):
    """Workgroups enough for every wavefront to have tiles of its own, short lists, and
    one expert that every token names."""
    def spoil(idx):
        idx[:, 3] = E // 2
        idx[0, :2] = E - 1
    check(*weights(fmt, group, zeros, E, H, I), N, 9, spoil=spoil)


@pytest.mark.parametrize("fmt,group,zeros", [("int4", 128, False), ("int4", 64, True),
                                             ("int4", 32, True), ("mxfp4", 32, False)])
def test_shared_x_of_long_lists(fmt, group, zeros):
    """The most pairs: about 115 tokens to each expert."""
    check(*weights(fmt, group, zeros, 64, 1024, 512), 256, 32)


@pytest.mark.parametrize("N", [13, 16])
@pytest.mark.parametrize("fmt,group,zeros", [("int4", 128, False), ("int4", 128, True)])
def test_shared_x_of_few_tokens(fmt, group, zeros, N):
    """Up to 16 tokens that name most experts, whole chunks of scales."""
    check(*weights(fmt, group, zeros, 258, 1024, 256), N, 31, absent=0.0)
