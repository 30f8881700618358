"""int4_cache_append's sum of squares: one order whichever form a call takes, so that a key's
code and a query's bits do not depend on how many rows came with it. The rows here are
binary32 ones made so that another order of the same sum gives another code."""
from fractions import Fraction

import numpy as np
import pytest
import torch

DEV = "cuda:0"


def squares_in_lanes(x):
    """8 channels a lane one after the other, then the lanes pair by pair (binary64; the square of a
    binary32 value is exact there, so that a fused product and a rounded one are the same)."""
    s = np.zeros(len(x) // 8)
    for e in range(8):
        s = s + x.reshape(-1, 8)[:, e].astype(np.float64) ** 2
    while len(s) > 1:
        s = s[0::2] + s[1::2]
    return s[0]


def squares_in_quads(x):
    """Four threads, each its channels 32 i + 8 a + e one after the other."""
    s = np.zeros(4)
    for i in range(len(x) // 32):
        for e in range(8):
            s = s + x.reshape(-1, 4, 8)[i, :, e].astype(np.float64) ** 2
    return (s[0] + s[1]) + (s[2] + s[3])


def factor(total, D):
    """binary32(1 / sqrt(total / D)) of a binary64 total, D a power of two, from whole numbers."""
    m = Fraction(total) / D
    r = np.float32(1.0 / np.sqrt(float(m)))
    for a in (np.nextafter(r, np.float32(0)), r, np.nextafter(r, np.float32(99))):
        b = np.nextafter(a, np.float32(99))
        low, high = (Fraction(float(a)) + Fraction(float(np.nextafter(a, np.float32(0))))) / 2, (Fraction(float(a)) + Fraction(float(b))) / 2
        if m * low * low < 1 <= m * high * high:
            return a
    raise AssertionError


def row_between(D):
    """A row whose sum lies next to where the factor's rounding turns: one large square and, in the same
    thread of four, small ones that vanish next to it one by one and not together."""
    x = np.zeros(D, np.float32)
    x[0] = 1.2
    at = np.array([32 * i + e for i in range(1, D // 32) for e in range(8)])
    x[at] = np.float32(np.sqrt(0.49 * 2.0 ** -52))                         # of a sum above 1: each less than half a step
    x[16], x[17] = 0.125, -0.125                                            # channels whose codes are looked at
    small = sum(Fraction(float(v)) ** 2 for v in x[at])
    known = Fraction(float(x[0])) ** 2 + 2 * Fraction(1, 64)
    # a turn of the factor: 1 / sqrt(m) halfway between two binary32 numbers, a little above what is there
    r = np.float32(1.0 / np.sqrt(float(known / D)))
    while True:
        r = np.nextafter(r, np.float32(0))
        mid = (Fraction(float(r)) + Fraction(float(np.nextafter(r, np.float32(99))))) / 2
        rest = D / (mid * mid) - small / 2 - known
        if rest > 0:
            break
    for d in (8, 9, 10):                                                    # the rest as squares, in another thread
        x[d] = np.float32(np.sqrt(float(rest)))
        if Fraction(float(x[d])) ** 2 > rest:
            x[d] = np.nextafter(x[d], np.float32(0))
        rest -= Fraction(float(x[d])) ** 2
    a, b = squares_in_lanes(x), squares_in_quads(x)
    # both sums are further from the turn than the factor's own error (2^-52, 2^-51 of the sum)
    turn = D / (mid * mid)
    assert Fraction(a) - turn > 2 * turn / 2 ** 52 and turn - Fraction(b) > 2 * turn / 2 ** 52
    return x, factor(a, D), factor(b, D)


def weight_between(x, r, other):
    """Weights for which channel 16's code is 1 with the larger factor's product below a half step, and 2 with
    the other: largest value of the group 7 steps, the channel on the border of 1.5."""
    w = np.ones(len(x), np.float32)
    w[0] = np.float32(7.0 / (x[0] * r))
    tops = [np.float32(np.float32(x[0] * f) * w[0]) for f in (r, other)]
    scales = [np.float32(np.float16(t / np.float32(7))) for t in tops]
    assert scales[0] == scales[1]
    border = np.float32(1.5) * scales[0]
    w[16] = np.float32(border / np.float32(x[16] * r))
    for _ in range(64):
        y = [np.float32(np.float32(x[16] * f) * w[16]) for f in (r, other)]
        if min(y) < border <= max(y):
            return w
        w[16] = np.nextafter(w[16], np.float32(99 if max(y) < border else 0))
    raise AssertionError


@pytest.mark.parametrize("D", [128, 256])
def test_rows_where_the_order_shows(D):
    """(no GPU) the two orders give two factors, and these two codes."""
    x, r, other = row_between(D)
    assert r != other
    w = weight_between(x, r, other)
    codes = []
    for f in (r, other):
        y = (x * f) * w
        codes.append(np.rint(y / np.float32(np.float16(np.abs(y).max() / np.float32(7)))))
    assert codes[0][16] != codes[1][16]


@pytest.mark.gpu
@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("turn", [None, "halves", "pairs"])
@pytest.mark.parametrize("D", [128, 256])
def test_codes_do_not_depend_on_the_form(D, turn, affine):
    """Rows by the hundred go row by row, by the ten thousand by positions."""
    import dequantizing_gemm_amd as dq
    x, r, other = row_between(D)
    w = torch.from_numpy(weight_between(x, r, other)).to(DEV)
    T, S = 2 ** 24 // D, 64
    assert 2 * T * D * 3 > 20000000 * 2
    g = torch.Generator(device=DEV).manual_seed(D)
    rows = torch.randn(T, 1, D, generator=g, device=DEV)
    rows[::97, 0] = torch.from_numpy(x).to(DEV)
    rope = None
    if turn:                                             # angle 0: the codes of the rows above stay what they are
        rope = torch.cat([torch.ones(T, D // 2, device=DEV), torch.zeros(T, D // 2, device=DEV)], 1)
    kw = dict(q_norm=w, k_norm=w, eps=0.0, rope=rope, interleaved=turn == "pairs")
    table = torch.arange(T // S, dtype=torch.int32, device=DEV)[None]
    caches = [dq.Int4Cache.empty(T // S, S, 1, D, D, affine) for _ in range(2)]
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    print("case: order", D, turn, affine, flush=True)
    whole = dq.int4_cache_append(caches[0], rows, rows, rows, table, i32(T), i32(0, T), **kw)
    for at in range(0, T, 16384):
        n = min(16384, T - at)
        part = dq.int4_cache_append(caches[1], rows[at:at + n], rows[at:at + n], rows[at:at + n], table, i32(at + n), i32(0, n), **kw)
        assert torch.equal(whole[at:at + n], part)
    for name in ("k_packed", "k_scales", "v_packed", "v_scales") + (("k_zeros", "v_zeros") if affine else ()):
        assert torch.equal(getattr(caches[0], name), getattr(caches[1], name)), name
