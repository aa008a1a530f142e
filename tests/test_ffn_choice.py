"""Which kernels the sizes of the GPU tests run in, from launches recorded without a device: a
kernel whose tests would go to another one after a change of the choice is named here."""
import random
import shutil

import pytest

from combine_ep_get_amd import build as libbuild
from tests import test_gpu_ffn as tg
from tests import test_gpu_ffn_int8 as ti
from tests import test_gpu_ffn_sizes as ts
from tests.launch_recorder import Recorder

pytestmark = pytest.mark.skipif(shutil.which(libbuild.HIPCC) is None, reason="hipcc not available")


@pytest.fixture(scope="module")
def rec(tmp_path_factory):
    return Recorder(str(tmp_path_factory.mktemp("recorder")))


def rows(rec, c):
    n = c["N"] * c["K"]
    if c.get("ll"):
        return rec.rows(n, c["E"], c["R"], c["ll"])
    return rec.rows(n, c["E"])


def names(launches):
    return [k for k, _, _ in launches]


def block(rec, c, int8=False):
    return names(rec.ffn(rows(rec, c), c["H"], c["I"], int8))


def gradient(rec, c):
    return names(rec.backward(rows(rec, c), c["H"], c["I"]))


def wide(form, epilogue, int8=False):
    return f"product_kernel<{form}, {epilogue}, {str(int8).lower()}>"


def small(form, epilogue, int8=False):
    return f"small_kernel<{form}, {epilogue}, {str(int8).lower()}>"


def few(epilogue, int8, tiles, rounds=False):
    return f"few_kernel<{epilogue}, {str(int8).lower()}, {tiles}, {str(rounds).lower()}>"


GATE, ROWS, GRAD, MATRIX = "StoreGate", "StoreRows", "StoreGateGrad", "StoreMatrix"


def test_every_kernel_is_reached(rec):
    seen = {"combine_backward_kernel"}
    for c in tg.SHAPES + ts.MANY + ts.MIDDLE:
        seen.update(block(rec, c) + gradient(rec, c))
    for c in ti.SHAPES + ti.SUB_BLOCKS:
        seen.update(block(rec, c, True))
    assert sorted(seen) == rec.kernels


def test_wide_tiles(rec):
    for c in ts.MANY:
        assert block(rec, c)[0] == wide(0, GATE), c
    for c in ts.MANY[:2] + ts.MANY[3:]:
        assert block(rec, c)[1] == wide(0, ROWS), c
        assert gradient(rec, c)[1] == wide(1, ROWS), c
    for c in (ts.MANY[2], ts.MANY[3]):                     # two steps; many
        assert gradient(rec, c)[0] == wide(1, GRAD), c
    for c in ts.MANY[3:]:
        assert gradient(rec, c)[2] == wide(2, MATRIX), c
    n = 25 * sum((0, 1, 64, 65, 127, 128, 129, 192, 255, 256, 257, 384, 385))
    for H, I in ((272, 144), (128, 64)):                   # tall tiles, then short ones
        for int8 in (False, True):
            got = names(rec.ffn(rec.rows(n, 325), H, I, int8))
            assert got[int8] == wide(0, GATE, int8) and got[-1] == wide(0, ROWS, int8)
    most = rec.rows(131072, 1024)
    assert names(rec.ffn(most, 256, 64)) == [wide(0, GATE), wide(0, ROWS)]
    assert names(rec.backward(most, 256, 64))[1:] == [wide(1, ROWS), wide(2, MATRIX)]


def test_middle_tiles(rec):
    for c in ts.MIDDLE:
        assert block(rec, c)[0] == small(0, GATE), c
        assert gradient(rec, c)[:2] == [small(1, GRAD), small(1, ROWS)], c
    assert block(rec, ts.MIDDLE[0])[1] == small(0, ROWS)
    for c in (ts.MANY[0], ts.MANY[1]):                     # 64 and 79 steps of an odd width
        assert gradient(rec, c)[2] == small(2, MATRIX), c


def test_low_latency(rec):
    for c, kernels in ((ti.SUB_BLOCKS[0], (few(GATE, False, 1), few(ROWS, False, 1))),
                       (ti.SUB_BLOCKS[1], (few(GATE, False, 2), few(ROWS, False, 2))),
                       (ti.SUB_BLOCKS[2], (small(0, GATE), small(0, ROWS))),
                       (ti.SUB_BLOCKS[5], (wide(0, GATE), wide(0, ROWS)))):
        assert tuple(block(rec, c)) == kernels, c
        assert tuple(block(rec, c, True)[1::2]) == tuple(k.replace("false", "true", 1)
                                                         for k in kernels), c


def test_int8(rec):
    kinds = [(0, few(GATE, True, 1), few(ROWS, True, 1)),
             (1, few(GATE, True, 1, True), few(ROWS, True, 1, True)),
             (2, few(GATE, True, 1, True), few(ROWS, True, 1, True)),
             (3, few(GATE, True, 1, True), few(ROWS, True, 1, True)),
             (4, few(GATE, True, 1), few(ROWS, True, 1)),
             *[(i, few(GATE, True, 2), few(ROWS, True, 2)) for i in (5, 6, 7)],
             *[(i, small(0, GATE, True), small(0, ROWS, True)) for i in (8, 9)],
             *[(i, wide(0, GATE, True), wide(0, ROWS, True)) for i in (10, 11, 12, 13)]]
    assert len(kinds) == len(ti.SHAPES)
    for i, *want in kinds:
        got = [k for k in block(rec, ti.SHAPES[i], True) if "quantize" not in k]
        assert got == want, ti.SHAPES[i]


def test_grids(rec):
    """Every launch has less than 2^32 threads along an axis (more would wrap, and be lost), and
    combine's gradient has a workgroup for each token."""
    rng = random.Random(5)
    drawn = [(rng.randrange(1, 1 << rng.randrange(1, 31)), rng.randrange(1, 1025),
              8 * rng.randrange(1, 1 << rng.randrange(1, 14))) for _ in range(300)]
    for N, K, H in [((1 << 26) + 5, 1, 8), (5000000, 1, 7168), (1 << 21, 32, 65536),
                    *[(n, 1 + k % 32, h) for n, k, h in drawn]]:
        if N * K > 2 ** 31 - 1:
            continue
        launches = rec.combine(N, K, H, N)
        assert sum(g[0] for _, g, _ in launches) == N
        for _, g, b in launches:
            assert g[0] * b[0] < 1 << 32 and g[1] == -(-K // 4) and b[1:] == (1, 1)
    for n, e, h in drawn:
        n, cols = min(n, 1 << 22), min(16 * (h // 16 + 1), 65536)
        for r in (rec.rows(n), rec.rows(n, e, capacity=max(n, 1 << 10))):
            for got in (rec.integer(r, cols, min(h, 4096)), rec.ffn(r, 512, 16 * (1 + h % 64)),
                        rec.backward(r, 512, 16 * (1 + h % 64)), rec.quantize(n, cols)):
                for _, g, b in got:
                    assert 0 < g[0] * b[0] < 1 << 32 and 0 < g[1] < 1 << 16
