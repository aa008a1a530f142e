"""The sizes that the experts' block and the 8-bit products refuse are those the header states:
on either side of each limit, on the host (device pointers here are made up)."""
import ctypes

import pytest

import combine_ep_get_amd as ep
from tests.test_ffn_abi import INT8, INVALID, accepted, no_gpu, weight

TOP = 2 ** 31 - 1
FAR = [i << 50 for i in range(1, 12)]        # farther apart than any buffer here is long


def ceil(a, b):
    return -(-a // b)


def stated(E, cap, cols):
    return ((cap // 16 + E) * ceil(cols, 16) <= TOP and E * cap // 16 + E <= TOP
            and (E * cap // 256 + E) * ceil(cols, 128) <= TOP - 1024)


def region(cap, E):
    return ep.RowsDesc(FAR[0], FAR[0] + (1 << 20), cap, E, 1, 0, 32)


def blocks(E, R, M):
    return ep.RowsDesc(None, FAR[0], E * R * M, E, R, M, 32)


def ffn(rows, H, I, int8=False):
    w = [weight(INT8, at, at + (1 << 49)) if int8 else weight(data=at) for at in FAR[1:3]]
    a = ep.FfnArgs(FAR[3], *w, FAR[4], None, FAR[5], H, I)
    return ep.lib().ep_ffn(ctypes.byref(rows), ctypes.byref(a), None)


def grad(rows, H, I):
    a = ep.FfnGradArgs(*FAR[1:10], H, I)
    return ep.lib().ep_ffn_backward(ctypes.byref(rows), ctypes.byref(a), None)


def integer(rows, C, O):
    a = ep.Int8Args(FAR[1], None, weight(INT8, FAR[2], FAR[3]), FAR[4], FAR[5], C, O)
    return ep.lib().ep_integer_linear(ctypes.byref(rows), ctypes.byref(a), None)


def edge(ok, top):
    """The largest n <= top with ok(n); ok(0) holds."""
    lo, hi = 0, top + 1
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if ok(mid) else (lo, mid)
    return lo


# which of the three binds: the second, the third, the first, none of them
@no_gpu
@pytest.mark.parametrize("E,H,I", [(1024, 16, 16), (1024, 64, 4096), (2, 32768, 32768), (1, 16, 8)])
def test_capacity(E, H, I):
    cols = max(H, 2 * I)
    cap = edge(lambda n: stated(E, n, cols), TOP)
    assert accepted(ffn(region(cap, E), H, I)) and accepted(grad(region(cap, E), H, I))
    assert accepted(integer(region(cap, E), 16, cols))
    if cap < TOP:
        assert ffn(region(cap + 1, E), H, I) == grad(region(cap + 1, E), H, I) == INVALID
        assert integer(region(cap + 1, E), 16, cols) == INVALID


@no_gpu
def test_sub_blocks():
    span = 0x60000000
    for H, I in ((7168, 2048), (2048, 7168)):
        M = (span - 1) // (2 * 7168 * 8)
        assert 8 * M * 2 * 7168 < span <= 8 * (M + 1) * 2 * 7168
        for int8 in (False, True):
            assert accepted(ffn(blocks(2, 8, M), H, I, int8))
            assert ffn(blocks(2, 8, M + 1), H, I, int8) == INVALID
    M = (span - 1) // (7168 * 8)
    assert accepted(integer(blocks(2, 8, M), 7168, 64))
    assert integer(blocks(2, 8, M + 1), 7168, 64) == INVALID
    assert accepted(ffn(region(1 << 20, 1), 7168, 2048))     # with offsets: any length


@no_gpu
def test_gradients_of_weights():
    E, H = 1024, 65536
    tiles = lambda i: E * (ceil(16 * i, 64) + ceil(8 * i, 64)) * ceil(H, 64)      # noqa: E731
    i = edge(lambda n: tiles(n) <= TOP - 1024, 65536 // 8)
    assert i < 65536 // 8
    assert accepted(grad(region(64, E), H, 8 * i))
    assert grad(region(64, E), H, 8 * (i + 1)) == INVALID


def test_sizes_beyond_32_bits(monkeypatch):
    """The binding refuses what ctypes would cut to 32 bits: 2^32 + 16 columns are not 16."""
    class Matrix:                            # of any size, without memory
        def __init__(self, *shape):
            self.shape = shape

        def get_device(self):
            return 0

        def data_ptr(self):
            return FAR[0]
        new_empty = checked_desc = lambda self, *a, **kw: self

    monkeypatch.setattr(ep, "_arg", lambda *a: None)
    monkeypatch.setattr(ep, "_call", lambda *a: pytest.fail("a call with sizes cut off"))
    wide, many, x = Matrix(1, 2 ** 32 + 16), Matrix(2 ** 32 + 1, 16), Matrix(1, 16)
    big = ep.Int8Weight.__new__(ep.Int8Weight)
    big.__dict__.update(shape=(2 ** 32 + 16, 16), codes=x, scales=x, desc=(FAR[0], FAR[0], 0, 3, 0))
    for call in (lambda: ep.quantize_int8(wide), lambda: ep.quantize_int8(many),
                 lambda: ep.expert_ffn(many, Matrix(32, 16), Matrix(16, 16)),
                 lambda: ep.expert_ffn(x, Matrix(2 ** 33 + 32, 16), Matrix(16, 2 ** 32 + 16),
                                       out=x),
                 lambda: ep.expert_ffn_backward(x, x, x, Matrix(2 ** 33 + 32, 16),
                                                Matrix(16, 2 ** 32 + 16), out=(x, x, x)),
                 lambda: ep.int8_linear(x, big, x_scales=x),
                 lambda: ep.ffn_workspace_bytes(4, 2 ** 32 + 64, 32),
                 lambda: ep.ffn_workspace_bytes(4, 64, -2 ** 32 + 32),
                 lambda: ep.ffn_workspace_bytes(2 ** 32 + 4, 64, 32),
                 lambda: ep.ep_integer_workspace_bytes(4, 2 ** 32 + 64)):
        with pytest.raises(ValueError):
            call()
