"""Attention over the 4-bit cache on MI355X where its arithmetic could leave its
range: scores of any size below 2^96, the smallest factors, value scales that are
far apart, hidden or negative. Bounds as in tests/test_cache_gpu.py unless a test
derives its own."""
import numpy as np
import pytest
import torch

from tests.cache_model import Model, plan
from tests.test_cache_gpu import BF16, DEV, F16, cache_of, check_attention, dev, dq, filled, rounded, say, values  # noqa: F401

pytestmark = pytest.mark.gpu


def two_level(dq, rng, D, group, affine, page, n, rows, tall, factors, dtype, scale, size=1.0):
    """A sequence of n tokens whose keys are zero but for those in `tall`, which are
    all the same: every score is 0 or the row's own S, from one dot product, so that
    the softmax weighs the visible keys of the larger one alike (for |S| of 2^20 and
    more the others are below e^(-2^20), which is 0). The last `rows` tokens are
    queries: one vector times a power of two of either sign each. `size` multiplies the
    values.

    Bounds: each weight is rounded to binary16 (2^-11), and the exponential, the sums
    and the division add 2^-20; the value sums round at 15 * 2^-24 of the scales for
    each 32 tokens, and the result once to its type. lse: the score's sum of D
    products in binary32, 2^-24 (D + 16) sum |q_d| 16 s, and 2^-22 of itself."""
    table, pages, _ = plan(rng, [n], [rows], page)
    m = Model(pages, page, 1, D, group, affine, fill=0x7E)
    whole = np.array([0, n], np.int32)
    q0 = rounded(rng.normal(size=D).astype(np.float32), dtype)
    k = np.zeros((n, 1, D), np.float32)
    k[sorted(tall)] = q0 * np.float32(0.25)
    m.write(k, values(rng, n, 1, D) * np.float32(size), table, [n], whole)
    vv = m.read(n, table, [n], whole)[1][:, 0].astype(np.float64)
    kk, ks = (x[0].astype(np.float64) for x in m.values("k", m.page(table, 0, min(tall)), min(tall) % page))
    vs = np.stack([m.values("v", m.page(table, 0, j), j % page)[1][0] for j in range(n)]).astype(np.float64)
    is_tall = np.isin(np.arange(n), sorted(tall))
    cache, table_d, lens = cache_of(dq, m), dev(table), dev(np.array([n], np.int32))
    for turn in range(0, len(factors), min(rows, len(factors))):
        q = (q0 * np.resize(np.roll(factors, -turn), rows)[:, None]).astype(np.float32)
        assert np.array_equal(rounded(q, dtype), q)
        out, lse = dq.int4_cache_attention(torch.from_numpy(q[:, None]).to(dtype).to(DEV), cache, table_d, lens,
                                           dev(np.array([0, rows], np.int32)), scale=scale, return_lse=True)
        torch.cuda.synchronize()
        o, l = out[:, 0].double().cpu().numpy(), lse[:, 0].double().cpu().numpy()
        assert np.all(np.isfinite(o)) and np.all(np.isfinite(l))
        for i in range(rows):
            S = scale * float(q[i].astype(np.float64) @ kk)
            assert 2.0 ** 20 <= abs(S) < 2.0 ** 96
            see = np.arange(n) <= n - rows + i
            best, level = see & is_tall, S
            if S < 0 and (see & ~is_tall).any() or not best.any():
                best, level = see & ~is_tall, 0.0
            ref = vv[best].mean(0)
            tol = (2.0 ** -11 + 2.0 ** -20) * np.abs(vv[best]).mean(0) + (see.sum() / 32 + 64) * 2.0 ** -24 * 15 * vs[see].max()
            tol = tol + torch.finfo(dtype).eps / 2 * (np.abs(ref) + tol) + (2.0 ** -25 if dtype == F16 else 0.0)
            assert np.all(np.abs(o[i] - ref) <= tol), (i, S, np.max(np.abs(o[i] - ref) / tol))
            want = level + np.log(best.sum())
            ltol = scale * 2.0 ** -24 * (D + 16) * 16 * float(ks @ np.abs(q[i].astype(np.float64))) if level else 0.0
            assert abs(l[i] - want) <= ltol + 2.0 ** -20 + 2.0 ** -22 * abs(want), (i, S, l[i], want)


FAR = [  # D, group, affine, page, tokens, rows, tokens with the tall key, dtype, scale
    (64, 64, False, 16, 1, 1, {0}, BF16, 0.125),
    (128, 128, False, 16, 40, 3, {2, 9, 20}, BF16, 0.125),
    (64, 64, True, 16, 300, 2, {7, 100, 290}, BF16, 0.125),
    (128, 32, True, 64, 2600, 2, {3, 1000, 2590}, BF16, 0.125),              # shared out over blocks
    (64, 64, False, 64, 9300, 1, {3, 1000, 5000, 9290}, BF16, 0.125),        # over more than 8
    (256, 128, True, 16, 1500, 3, {1, 700, 1490}, BF16, 0.125),
    (64, 64, False, 32, 330, 300, {40, 41, 200}, BF16, 0.125),               # the form for prompts
    (128, 64, True, 32, 2300, 290, {2020, 2100, 2299}, BF16, 0.125),         # the same, shared out
    (192, 192, False, 32, 330, 300, {40, 41, 200}, BF16, 0.125),
    (64, 64, False, 16, 200, 5, {3, 77, 190}, F16, 2.0 ** 70),
]


@pytest.mark.parametrize("D,group,affine,page,n,rows,tall,dtype,scale", FAR)
def test_scores_far_from_zero(dq, D, group, affine, page, n, rows, tall, dtype, scale):
    factors = [2.0 ** 20, -2.0 ** 26, 2.0 ** 30, 2.0 ** 25, -2.0 ** 90, 2.0 ** 40, 2.0 ** 90, -2.0 ** 28, 2.0 ** 27,
               2.0 ** 21, -2.0 ** 21, 2.0 ** 22, -2.0 ** 23, 2.0 ** 24]
    if dtype == F16:
        factors = [1.0, -32.0, 256.0, 4.0]
    say("case: far", D, group, affine, page, n, rows, dtype, scale)
    two_level(dq, np.random.default_rng(70 + n), D, group, affine, page, n, rows, tall, factors, dtype, scale)
    if dtype == BF16:                      # value scales up to some thousands, without the room that small ones leave
        two_level(dq, np.random.default_rng(71 + n), D, group, affine, page, n, rows, tall, factors, dtype, scale, 2.0 ** 12)


SMALL = [(64, 64, False, 2, [70, 1, 33], [1, 1, 1]), (128, 32, True, 2, [1300, 20], [3, 1]), (64, 64, False, 3, [230, 290], [140, 290])]


@pytest.mark.parametrize("D,group,affine,ratio,lengths,new", SMALL)
def test_smallest_scales(dq, D, group, affine, ratio, lengths, new):
    """Products of scale and query down to the smallest binary32 numbers and below,
    where all visible keys weigh the same; some are hidden in each tile."""
    rng = np.random.default_rng(80 + D)
    m, table, starts = filled(rng, 1, D, group, affine, 16, lengths, new)
    q = rounded(rng.normal(size=(int(starts[-1]), ratio, D)).astype(np.float32), BF16)
    cache = cache_of(dq, m)
    st = None if set(new) == {1} else starts
    for scale in (1e-45, 1e-42, 2.0 ** -126):
        say("case: small scale", D, scale)
        check_attention(dq, m, table, lengths, st, q, BF16, scale=scale, cache=cache)
    tiny = rounded(q * np.float32(2.0 ** -120) * np.float32(2.0 ** -8), BF16)      # subnormal in binary32 as in bfloat16
    assert np.any(tiny) and np.abs(tiny).max() < 2.0 ** -125
    for scale in (2.0 ** -11, 2.0 ** -126, 1.0):
        say("case: small queries", D, scale)
        check_attention(dq, m, table, lengths, st, tiny, BF16, scale=scale, cache=cache)


@pytest.mark.parametrize("rows", [1, 300])
def test_largest_scales(dq, rows):
    """Products of scale and query beyond binary32, over keys that are all zero."""
    rng = np.random.default_rng(85)
    n = rows + 20
    table, pages, _ = plan(rng, [n], [rows], 16)
    m = Model(pages, 16, 1, 64, 64, False, fill=0x7E)
    m.write(np.zeros((n, 1, 64), np.float32), values(rng, n, 1, 64), table, [n], np.array([0, n], np.int32))
    q = rounded((rng.normal(size=(rows, 2, 64)) * 2.0 ** 96).astype(np.float32), BF16)
    say("case: large scale", rows)
    check_attention(dq, m, table, [n], np.array([0, rows], np.int32), q, BF16, scale=3e38)


@pytest.mark.parametrize("D,group,affine,ratio,rows,dtype", [
    (64, 64, False, 2, 14, BF16), (128, 64, True, 1, 30, F16), (128, 128, False, 2, 200, F16), (64, 32, True, 3, 140, BF16),
    (256, 128, False, 1, 20, BF16)])
def test_hidden_tokens_scales(dq, D, group, affine, ratio, rows, dtype):
    """Rows before a token whose value scales are far above theirs, in the same unit of
    16: what a row does not see takes no bits from what it sees."""
    rng = np.random.default_rng(90 + D + rows)
    n = rows + 20
    for low, high, at in ((2.0 ** -13, 2.0 ** 11, n - 1), (2.0 ** -17, 2.0 ** 5, n - 2), (2.0 ** -9, 2.0 ** 13, n - rows + 5)):
        table, pages, _ = plan(rng, [n], [rows], 16)
        m = Model(pages, 16, 1, D, group, affine, fill=0x7E)
        v = rng.normal(size=(n, 1, D)).astype(np.float32) * np.float32(low)
        v[at] *= np.float32(high / low)
        m.write(values(rng, n, 1, D), v, table, [n], np.array([0, n], np.int32))
        q = rounded(rng.normal(size=(rows, ratio, D)).astype(np.float32), dtype)
        say("case: hidden scales", D, rows, low, high)
        check_attention(dq, m, table, [n], np.array([0, rows], np.int32), q, dtype)


@pytest.mark.parametrize("D,group,affine,rows,dtype", [(64, 64, False, 1, F16), (128, 32, True, 4, BF16), (128, 128, False, 300, F16)])
def test_any_bits_before_the_window(dq, D, group, affine, rows, dtype):
    """Tokens before every row's window may hold any bits, negative and NaN scales of
    either sign among them."""
    rng = np.random.default_rng(100 + D)
    n, window = rows + 60, 21
    m, table, _ = filled(rng, 1, D, group, affine, 16, [n], [rows])
    q = rounded(rng.normal(size=(rows, 2, D)).astype(np.float32), dtype)
    starts = np.array([0, rows], np.int32)
    for j in range(n - rows - window + 1):
        page, slot = m.page(table, 0, j), j % 16
        for s in "kv":
            bits = rng.integers(0, 65536, size=m.scales[s][page, :, slot // 16, :, slot % 16].shape).astype(np.uint16)
            m.scales[s][page, :, slot // 16, :, slot % 16] = (bits | 0x7C00 if j % 3 else bits).view(np.float16)
            if affine:
                m.zeros[s][page, :, slot // 16, :, slot % 16] = rng.integers(0, 256)
    say("case: any bits", D, rows)
    with np.errstate(invalid="ignore", over="ignore"):
        check_attention(dq, m, table, [n], starts, q, dtype, window=window)


@pytest.mark.parametrize("D,group,affine,lengths,new", [
    (64, 64, False, [40, 130], [1, 1]), (128, 64, True, [70, 2100], [3, 1]), (128, 128, False, [300, 20], [290, 20]),
    (256, 128, True, [50], [20])])
def test_negative_scales(dq, D, group, affine, lengths, new):
    """A cache filled elsewhere may hold a group's codes and scale both negated (the
    distances from the zero point, with affine codes): the same values."""
    rng = np.random.default_rng(110 + D)
    m, table, starts = filled(rng, 2, D, group, affine, 16, lengths, new)
    cache = cache_of(dq, m)
    for s in "kv":
        flip = torch.rand(m.scales[s].shape, device=DEV) < 0.5                   # [pages, heads, units, G, 16]
        if not affine:                                                           # -8 has no opposite
            codes = m.packed["v"] if s == "v" else np.take(m.packed["k"], np.argsort(m.key_order()), -1).reshape(
                m.P, 2, 1, 16, -1).transpose(0, 1, 2, 4, 3)
            eight = np.stack([(codes & 15) == 8, codes >> 4 == 8], -2).reshape(m.P, 2, 1, -1, 16)
            any8 = np.stack([eight[..., g * m.group:(g + 1) * m.group, :].any(-2) for g in range(m.G)], -2)
            flip &= ~dev(any8)
        scales, packed = getattr(cache, s + "_scales"), getattr(cache, s + "_packed")
        scales.copy_(torch.where(flip, -scales, scales))
        channel = flip.repeat_interleave(m.group, 3)[..., :D, :]                 # [pages, heads, units, D, 16]
        channel = torch.nn.functional.pad(channel, (0, 0, 0, 32 * m.C - D))
        low, high = channel[..., 0::2, :], channel[..., 1::2, :]                 # of each byte
        if s == "k":
            order = torch.from_numpy(m.key_order()).to(DEV)
            low, high = (x.transpose(-1, -2)[..., order].reshape(packed.shape) for x in (low, high))
        lo, hi = packed & 15, packed >> 4
        if affine:
            zeros = getattr(cache, s + "_zeros")
            zeros.copy_(torch.where(flip, 15 - zeros, zeros))
            lo, hi = torch.where(low, 15 - lo, lo), torch.where(high, 15 - hi, hi)
        else:
            lo, hi = torch.where(low, (16 - lo) & 15, lo), torch.where(high, (16 - hi) & 15, hi)
        packed.copy_(lo | hi << 4)
    say("case: negative scales", D, group, affine)
    whole = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    kr, vr, _ = m.read(int(whole[-1]), table, lengths, whole)
    kg, vg = dq.int4_cache_read(cache, dev(table), dev(np.array(lengths, np.int32)), dev(whole), rows=int(whole[-1]),
                                dtype=torch.float32)
    assert np.array_equal(kg.cpu().numpy(), kr) and np.array_equal(vg.cpu().numpy(), vr)
    q = rounded(rng.normal(size=(int(starts[-1]), 4, D)).astype(np.float32), BF16)
    check_attention(dq, m, table, lengths, None if set(new) == {1} else starts, q, BF16, cache=cache)


@pytest.mark.parametrize("gap", [2.0 ** -20, 2.0 ** -30])
@pytest.mark.parametrize("D,group,affine,n,rows", [(64, 64, False, 70, 1), (128, 128, True, 1500, 2), (128, 64, False, 300, 290)])
def test_value_scales_far_apart(dq, D, group, affine, n, rows, gap):
    """The first token of each unit of 16 takes nearly all the weight, with values far
    below the others': each product of probability p and scale s is rounded by 2^-11 of
    itself or by 2^-33 P max(S, 2^-15), P and S the largest among the visible tokens,
    whichever is more, and multiplies a code up to 15. Beside that, as in the model: the
    scores' roundings (delta, on every weight) and the sums'."""
    rng = np.random.default_rng(120 + D)
    table, pages, _ = plan(rng, [n], [rows], 16)
    m = Model(pages, 16, 1, D, group, affine, fill=0x7E)
    whole, starts = np.array([0, n], np.int32), np.array([0, rows], np.int32)
    q0 = rng.normal(size=D).astype(np.float32)
    k, v = rng.normal(size=(2, n, 1, D)).astype(np.float32) * np.array([1.0, 2.0 ** 14], np.float32)[:, None, None, None]
    k[:, 0] -= np.outer(k[:, 0] @ q0, q0) / (q0 @ q0)
    k[::16] = q0 * np.float32(50.0 * np.sqrt(D) / (q0 @ q0))       # scores of 50 against about 1
    v[::16] *= np.float32(gap)
    m.write(k, v, table, [n], whole)
    q = rounded(np.repeat(q0[None, None], rows, 0), BF16)
    say("case: far apart", D, n, rows, gap)
    out = dq.int4_cache_attention(torch.from_numpy(q).to(BF16).to(DEV), cache_of(dq, m), dev(table), dev(np.array([n], np.int32)),
                                  dev(starts)).double().cpu().numpy()[:, 0]
    at = [(m.page(table, 0, j), j % 16) for j in range(n)]
    kk, ks = (np.array([m.values("k", *x)[i][0] for x in at], np.float64) for i in (0, 1))
    vv, vs = (np.array([m.values("v", *x)[i][0] for x in at], np.float64) for i in (0, 1))
    for i in range(rows):
        see, x = np.arange(n) <= n - rows + i, q[i, 0].astype(np.float64)
        a = kk[see] @ x * D ** -0.5
        p = np.exp(a - a.max())[:, None]
        p /= p.sum()
        ref = (p * vv[see]).sum(0)
        delta = (D ** -0.5 * 2.0 ** -24 * (D + 16) * (16 * ks[see] @ np.abs(x)) + 2.0 ** -22 * np.abs(a)).max()
        once = np.maximum(2.0 ** -11 * p * vs[see], 2.0 ** -33 * p.max() * np.maximum(vs[see].max(), 2.0 ** -15))
        bound = 15 * (once * (vv[see] != 0)).sum(0) + (2 * delta + 2.0 ** -20) * (p * np.abs(vv[see])).sum(0)
        bound += (see.sum() / 32 + 64) * 2.0 ** -24 * 15 * (p * vs[see]).sum(0)
        bound += torch.finfo(BF16).eps / 2 * (np.abs(ref) + bound)
        assert np.all(np.abs(out[i] - ref) <= bound), (i, np.max(np.abs(out[i] - ref) / bound))
