"""gate_up of the experts' block on the sub-blocks of the low-latency dispatch."""
import pytest

import combine_ep_get_amd as ep
from tests.test_gpu_ffn import Case, check_ffn, ident
from tests.test_gpu_ffn_int8 import SUB_BLOCKS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", SUB_BLOCKS, ids=ident)
def test_gate_up(shape):
    c = Case(91, **shape)
    y, gu = c.full(c.H), c.full(2 * c.I)
    ep.expert_ffn(c.x, c.w13, c.w2, layout=c.layout, out=y, gate_up=gu)
    c.untouched(y)
    c.untouched(gu)
    check_ffn(c, y, gu)
