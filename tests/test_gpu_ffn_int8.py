"""The experts' block with 8-bit weights value by value, with gate_up, on every kind of rows and
in every kernel that its products run in (tests/test_ffn_choice.py holds that)."""
import pytest
import torch

import combine_ep_get_amd as ep
from tests import ffn_tight as tight
from tests.test_gpu_ffn import Case, ident

pytestmark = pytest.mark.gpu

SHAPES = [
    dict(N=1, K=1, E=1, A=1, H=16, I=16, drop=0),
    dict(N=1, K=1, E=0, A=1, H=2048, I=1024),                     # rounded on the way
    dict(N=7, K=1, E=0, A=1, H=1040, I=528),
    dict(N=16, K=1, E=0, A=1, H=1024, I=1008),
    dict(N=64, K=1, E=64, A=1, H=64, I=80, skew=3.0),             # 16 rows a tile
    dict(N=37, K=2, E=5, A=4, H=144, I=80),                       # 32 rows a tile
    dict(N=300, K=3, E=7, A=16, H=272, I=208, skew=2.0),
    dict(N=257, K=1, E=0, A=1, H=1008, I=352),
    dict(N=700, K=2, E=3, A=128, H=512, I=272, drop=0.4),         # 64-row tiles
    dict(N=333, K=1, E=0, A=1, H=4080, I=2064),
    dict(N=4096, K=1, E=0, A=1, H=1024, I=512),                   # 256-row tiles
    dict(N=6000, K=1, E=0, A=1, H=1008, I=528),
    dict(N=3000, K=3, E=4, A=16, H=1008, I=528, skew=1.0),
    dict(N=3000, K=2, E=40, A=1, H=1072, I=272, skew=0.7),        # and those of 128 rows
]
SUB_BLOCKS = [
    dict(N=8, K=2, E=4, A=1, H=64, I=32, R=2, ll=4),
    dict(N=48, K=3, E=12, A=1, H=272, I=144, R=4, ll=12),
    dict(N=256, K=8, E=32, A=1, H=512, I=256, R=8, ll=32),
    dict(N=600, K=2, E=2, A=1, H=128, I=64, R=2, ll=300, drop=0),
    dict(N=400, K=2, E=4, A=1, H=2064, I=1040, R=4, ll=100),
    dict(N=4000, K=2, E=8, A=1, H=1008, I=528, R=8, ll=500),
]


@pytest.mark.parametrize("shape", SHAPES + SUB_BLOCKS, ids=ident)
def test_block(shape):
    c = Case(81, int8=True, **shape)
    y, gu = c.full(c.H), c.full(2 * c.I)
    ep.expert_ffn(c.x, c.w13, c.w2, layout=c.layout, out=y, gate_up=gu)
    c.untouched(y)
    c.untouched(gu)
    for e, s in c.where:
        if len(s) == 0:
            continue
        w = [(w.codes, w.scales) if e is None else (w.codes[e], w.scales[e]) for w in (c.w13, c.w2)]
        want, choices = tight.block(c.x[s], *w)
        tight.check_gate_up(gu[s], want, f"gate_up of expert {e}")
        tight.check_rows(y[s], choices, f"y of expert {e}")
    again = ep.expert_ffn(c.x, c.w13, c.w2, layout=c.layout)      # without gate_up
    assert torch.equal(again[c.at], y[c.at])
