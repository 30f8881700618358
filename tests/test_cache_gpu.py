"""The 4-bit key/value cache on MI355X against the plain model of
tests/cache_model.py: written bytes and values read back must match it bit for
bit, attention must stay within the bound derived there plus half a step of the
output's type."""
import numpy as np
import pytest
import torch

from tests.cache_model import Model, plan

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def dq():
    import dequantizing_gemm_amd as dq
    return dq


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def say(*a):
    print(*a, flush=True)


def cache_of(dq, m):
    """An Int4Cache with a model's contents."""
    return dq.Int4Cache(dev(m.packed["k"]), dev(m.scales["k"]), dev(m.packed["v"]), dev(m.scales["v"]), m.D, m.group,
                        *(dev(m.zeros[s]) if m.affine else None for s in "kv"))


def assert_same_bytes(cache, m):
    torch.cuda.synchronize()
    for s in "kv":
        assert np.array_equal(getattr(cache, s + "_packed").cpu().numpy(), m.packed[s]), f"{s} codes"
        assert np.array_equal(getattr(cache, s + "_scales").cpu().numpy().view(np.uint16),
                              m.scales[s].view(np.uint16)), f"{s} scales"
        if m.affine:
            assert np.array_equal(getattr(cache, s + "_zeros").cpu().numpy(), m.zeros[s]), f"{s} zeros"


def values(rng, *shape):
    x = rng.normal(size=shape).astype(np.float32)
    return x * np.exp(0.7 * rng.normal(size=shape[-1:])).astype(np.float32)


def rounded(x, dtype):
    """float32 values that dtype holds exactly."""
    return torch.from_numpy(x).to(dtype).float().numpy()


def filled(rng, heads, D, group, affine, page, lengths, new, spare=3):
    """A model whose sequences hold random keys and values, and its plan."""
    table, pages, starts = plan(rng, lengths, new, page, spare)
    m = Model(pages, page, heads, D, group, affine, fill=0x7E)   # NaN scales where nothing was written
    whole = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    T = int(whole[-1])
    m.write(values(rng, T, heads, D), values(rng, T, heads, D), table, np.asarray(lengths), whole)
    return m, table, starts


def check_attention(dq, m, table, lengths, starts, q, dtype, *, scale=None, causal=True, window=0, rows=None, cache=None,
                    **kw):
    """One call against the model; q float32 [rows, Hq, D] holds values of dtype."""
    cache = cache or cache_of(dq, m)
    scale_used = m.D ** -0.5 if scale is None else scale
    qd = torch.from_numpy(q).to(DEV).to(dtype)
    mark = torch.full(qd.shape, 7.0, dtype=dtype, device=DEV)
    out, lse = dq.int4_cache_attention(qd, cache, dev(table), dev(np.asarray(lengths, np.int32)),
                                       None if starts is None else dev(starts), scale=scale, causal=causal,
                                       window=window, return_lse=True, out=mark, **kw)
    torch.cuda.synchronize()
    ref, rlse, owned, tol, ltol = m.attend(q, table, np.asarray(lengths), starts, scale_used, causal, window)
    o, l = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    assert np.all(o[~owned] == 7.0), "a row that no sequence owns was written"
    tol = tol + torch.finfo(dtype).eps / 2 * (np.abs(ref) + tol) + (2.0 ** -25 if dtype == F16 else 0.0)
    err = np.abs(o - ref)[owned]
    assert np.all(np.isfinite(o[owned]))
    assert np.all(err <= tol[owned]), f"worst error / bound {np.max(err / np.maximum(tol[owned], 1e-30))}"
    none = np.isneginf(rlse) & owned[:, None]
    assert np.all(np.isneginf(l[none])) and np.all(o[none] == 0)
    some = owned[:, None] & ~none
    lerr = np.abs(l[some] - rlse[some])
    assert np.all(lerr <= ltol[some]), f"lse: worst error / bound {np.max(lerr / ltol[some])}"
    return out, lse


# ---------------------------------------------------------------- write, read

STORE = [  # D, group, affine, heads, page, dtype, lengths, new rows
    (128, 128, False, 2, 16, BF16, [1, 17, 40], [1, 17, 33]),
    (128, 64, True, 3, 32, F16, [5, 64, 33, 0], [5, 30, 1, 0]),
    (128, 32, False, 1, 64, F32, [200], [150]),
    (64, 64, True, 4, 16, BF16, [31, 2], [31, 1]),
    (64, 32, False, 2, 128, F16, [129, 128], [3, 128]),
    (80, 32, True, 2, 16, F32, [19, 1, 50], [19, 1, 7]),
    (72, 128, False, 1, 16, BF16, [33], [33]),
    (96, 64, False, 2, 32, BF16, [40, 70], [11, 70]),
    (192, 128, True, 2, 16, F16, [21, 20], [21, 3]),
    (256, 128, False, 1, 32, BF16, [65, 9], [64, 9]),
    (256, 32, True, 2, 16, F16, [18], [18]),
    (160, 256, False, 2, 16, F32, [17], [17]),
    (1, 1, False, 2, 16, F32, [5], [5]),
    (33, 32, True, 1, 16, BF16, [20], [20]),
    (250, 64, False, 1, 16, F16, [16], [16]),
]


@pytest.mark.parametrize("D,group,affine,heads,page,dtype,lengths,new", STORE)
def test_write_and_read(dq, D, group, affine, heads, page, dtype, lengths, new):
    rng = np.random.default_rng(D + group)
    table, pages, starts = plan(rng, lengths, new, page)
    m = Model(pages, page, heads, D, group, affine, fill=0x5A)
    cache = cache_of(dq, m)
    T = int(starts[-1])
    k, v = rounded(values(rng, T, heads, D), dtype), rounded(values(rng, T, heads, D), dtype)
    k[0], v[T // 2] = 0.0, 0.0                                  # groups of zeros
    say("case: write", D, group, affine, dtype, T)
    # keys and values as slices of one fused projection
    fused = torch.from_numpy(np.stack([k, v], 1)).to(DEV).to(dtype)
    dq.int4_cache_write(cache, fused[:, 0], fused[:, 1], dev(table), dev(np.asarray(lengths, np.int32)), dev(starts))
    m.write(k, v, table, np.asarray(lengths), starts)
    assert_same_bytes(cache, m)
    kr, vr, owned = m.read(T, table, np.asarray(lengths), starts)
    assert owned.all()
    for out in (F32, F16, BF16):
        kg, vg = dq.int4_cache_read(cache, dev(table), dev(np.asarray(lengths, np.int32)), dev(starts), rows=T, dtype=out)
        assert torch.equal(kg.cpu(), torch.from_numpy(kr).to(out)) and torch.equal(vg.cpu(), torch.from_numpy(vr).to(out))


def test_write_matches_the_weight_quantizer(dq):
    """A token's codes are quantize_int4's of its channels as one weight row."""
    torch.manual_seed(0)
    H, D = 4, 128
    cache = dq.Int4Cache.empty(1, 16, H, D, 64)
    k = torch.randn(16, H, D, device=DEV)
    dq.int4_cache_write(cache, k, k, torch.zeros(1, 1, dtype=torch.int32, device=DEV),
                        torch.tensor([16], dtype=torch.int32, device=DEV),
                        torch.tensor([0, 16], dtype=torch.int32, device=DEV))
    packed, scales, K = dq.quantize_int4(k.reshape(16 * H, D), 64)
    want = dq.dequantize_int4(packed, scales, K, 64, torch.float32).reshape(16, H, D)
    got = dq.int4_cache_read(cache, torch.zeros(1, 1, dtype=torch.int32, device=DEV),
                             torch.tensor([16], dtype=torch.int32, device=DEV),
                             torch.tensor([0, 16], dtype=torch.int32, device=DEV), rows=16, dtype=torch.float32)
    assert torch.equal(got[0], want) and torch.equal(got[1], want)


@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_write_strides_and_alignment(dq, dtype, offset):
    """Heads outermost, an odd base address, rows repeated by a zero stride."""
    rng = np.random.default_rng(offset)
    H, D, T = 3, 72, 21
    table, pages, starts = plan(rng, [T], [T], 16)
    m = Model(pages, 16, H, D, 72, False)
    cache = cache_of(dq, m)
    k, v1 = rounded(values(rng, T, H, D), dtype), rounded(values(rng, 1, H, D), dtype)
    buf = torch.zeros(H * T * D + offset, dtype=dtype, device=DEV)
    kd = buf[offset:].view(H, T, D).transpose(0, 1)
    kd.copy_(torch.from_numpy(k))
    vd = torch.from_numpy(v1).to(DEV).to(dtype).expand(T, H, D)
    dq.int4_cache_write(cache, kd, vd, dev(table), dev(np.array([T], np.int32)), dev(starts))
    m.write(k, np.repeat(v1, T, 0), table, [T], starts)
    assert_same_bytes(cache, m)


def bad_plan(rng, page):
    """Sequences with pages out of range, more rows than tokens, lengths past the
    table, negative and zero lengths; rows before and behind all sequences."""
    lengths = np.array([40, 3, 60, -5, 0, 47], np.int32)
    new = [20, 7, 12, 2, 3, 47]                    # the second: four rows before position 0
    table, pages, starts = plan(rng, np.maximum(lengths, 0), new, page)
    table = table[:, :3].copy()                    # 60 tokens: the last page is missing
    table[0, 1] = pages + 5
    table[5, 0] = -7
    table[5, 2] = 2 ** 31 - 1
    return table, pages, lengths, (starts + 2).astype(np.int32), int(starts[-1]) + 6


def test_write_and_read_bad_plans(dq):
    rng = np.random.default_rng(5)
    H, D = 2, 64
    table, pages, lengths, starts, T = bad_plan(rng, 16)
    m = Model(pages, 16, H, D, 64, True, fill=0x11)
    cache = cache_of(dq, m)
    k, v = values(rng, T, H, D), values(rng, T, H, D)
    dq.int4_cache_write(cache, dev(k), dev(v), dev(table), dev(lengths), dev(starts))
    m.write(k, v, table, lengths, starts)
    assert_same_bytes(cache, m)
    mark = (torch.full((T, H, D), 7.0, device=DEV), torch.full((T, H, D), 7.0, device=DEV))
    got = dq.int4_cache_read(cache, dev(table), dev(lengths), dev(starts), dtype=F32, out=mark)
    kr, vr, owned = m.read(T, table, lengths, starts)
    assert not owned.all()
    for g, r in zip(got, (kr, vr)):
        r[~owned] = 7.0
        assert np.array_equal(g.cpu().numpy(), r)


def test_extreme_values(dq):
    """Scales from the smallest binary16 to the largest, affine and symmetric."""
    rng = np.random.default_rng(6)
    H, D, T = 1, 128, 48
    x = values(rng, T, H, D) * np.exp2(rng.integers(-30, 12, size=(T, H, 1))).astype(np.float32)
    x[3, 0, :] = -8.0 * 2.0 ** -24
    x[4, 0, 5] = 7 * 65504.0
    for affine in (False, True):
        table, pages, starts = plan(rng, [T], [T], 16)
        m = Model(pages, 16, H, D, 32, affine)
        cache = cache_of(dq, m)
        dq.int4_cache_write(cache, dev(x), dev(-x), dev(table), dev(np.array([T], np.int32)), dev(starts))
        m.write(x, -x, table, [T], starts)
        assert_same_bytes(cache, m)


# ---------------------------------------------------------------- attention

ATTEND = [  # D, group, affine, heads, ratio, page, dtype, lengths, new rows, window
    (128, 128, False, 2, 4, 64, BF16, [1, 63, 64, 65, 300], [1] * 5, 0),
    (128, 64, False, 2, 4, 16, F16, [7, 1000], [1, 1], 0),
    (128, 32, True, 1, 8, 32, BF16, [515, 16, 17], [1] * 3, 0),
    (128, 128, True, 1, 16, 16, F16, [33, 257], [1, 1], 0),
    (64, 64, False, 3, 1, 16, F16, [1, 40, 129], [1] * 3, 0),
    (64, 32, True, 1, 20, 32, BF16, [90], [1], 0),
    (96, 96, False, 1, 6, 16, F16, [100, 31], [5, 31], 0),
    (96, 64, True, 1, 3, 16, BF16, [70], [9], 0),
    (80, 128, False, 2, 5, 16, BF16, [130, 20], [3, 20], 17),
    (72, 32, True, 1, 2, 16, F16, [60], [60], 0),
    (192, 64, False, 1, 4, 32, BF16, [140, 65], [2, 1], 0),
    (192, 128, True, 1, 1, 16, F16, [50], [50], 10),
    (256, 128, False, 1, 8, 32, BF16, [200, 33], [4, 33], 0),
    (256, 256, True, 1, 2, 16, F16, [90], [1], 0),
    (256, 32, False, 1, 4, 16, BF16, [70], [20], 0),
    (128, 128, False, 1, 4, 64, BF16, [333], [333], 0),
    (128, 128, False, 1, 4, 64, F16, [400, 90], [200, 90], 64),
    (160, 160, False, 1, 3, 16, F16, [45], [45], 0),
    (33, 33, False, 1, 2, 16, BF16, [20], [20], 0),
    (1, 1, True, 1, 1, 16, F16, [30], [2], 0),
    (128, 32, False, 1, 5, 16, F16, [150, 0, 80, 2], [1, 0, 80, 2], 0),
    (64, 64, True, 2, 2, 256, BF16, [700], [70], 100),
]


@pytest.mark.parametrize("D,group,affine,heads,ratio,page,dtype,lengths,new,window", ATTEND)
def test_attention(dq, D, group, affine, heads, ratio, page, dtype, lengths, new, window):
    rng = np.random.default_rng(D * 7 + group + sum(lengths))
    say("case: attention", D, group, affine, heads, ratio, page, dtype, lengths, new, window)
    m, table, starts = filled(rng, heads, D, group, affine, page, lengths, new)
    q = rounded(rng.normal(size=(int(starts[-1]), heads * ratio, D)).astype(np.float32), dtype)
    check_attention(dq, m, table, lengths, None if set(new) == {1} else starts, q, dtype, window=window)


def test_attention_without_causal_and_other_scale(dq):
    rng = np.random.default_rng(11)
    lengths, new = [150, 37], [20, 9]
    m, table, starts = filled(rng, 2, 64, 32, False, 16, lengths, new)
    q = rounded(rng.normal(size=(29, 4, 64)).astype(np.float32), BF16)
    check_attention(dq, m, table, lengths, starts, q, BF16, causal=False)
    check_attention(dq, m, table, lengths, starts, q, BF16, scale=0.3)


def test_attention_bad_plans_and_padded_batch(dq):
    """Rows without keys, pages out of range in the middle of a sequence (whose
    slots hold NaN scales), rows before and behind all sequences."""
    rng = np.random.default_rng(12)
    for affine in (False, True):
        table, pages, lengths, starts, T = bad_plan(rng, 16)
        m = Model(pages, 16, 2, 64, 32, affine, fill=0x7E)
        whole = np.concatenate([[0], np.cumsum(np.maximum(lengths, 0))]).astype(np.int32)
        n = int(whole[-1])
        m.write(values(rng, n, 2, 64), values(rng, n, 2, 64), table, np.maximum(lengths, 0), whole)
        q = rounded(rng.normal(size=(T, 6, 64)).astype(np.float32), F16)
        check_attention(dq, m, table, lengths, starts, q, F16)
        check_attention(dq, m, table, lengths, starts, q, F16, window=9)
        check_attention(dq, m, table, lengths, starts, q, F16, causal=False)


def test_attention_nothing_cached(dq):
    rng = np.random.default_rng(13)
    m = Model(2, 16, 1, 64, 64, False, fill=0x7E)
    q = rounded(rng.normal(size=(3, 2, 64)).astype(np.float32), F16)
    table = np.full((3, 1), -1, np.int32)
    check_attention(dq, m, table, [0, 0, 0], None, q, F16)
    check_attention(dq, m, table, [5, 16, 1], None, q, F16)          # lengths, but no pages
    check_attention(dq, m, table[:, :0], [5, 16, 1], None, q, F16)   # not even a table


def test_attention_poison_behind_the_rows(dq):
    """Tokens after a row's position and before its window may hold infinite or
    NaN scales."""
    rng = np.random.default_rng(14)
    n = 200
    m, table, _ = filled(rng, 1, 128, 64, True, 16, [n], [n])
    for j in list(range(0, 40)) + list(range(150, n)):
        page, slot = m.page(table, 0, j), j % 16
        for s in "kv":
            m.scales[s][page, :, slot // 16, :, slot % 16] = [np.inf, np.nan][j % 2]
            m.zeros[s][page, :, slot // 16, :, slot % 16] = 255
    cache = cache_of(dq, m)
    q = rounded(rng.normal(size=(n, 4, 128)).astype(np.float32), BF16)
    with np.errstate(invalid="ignore"):
        out, lse = dq.int4_cache_attention(torch.from_numpy(q).to(DEV).to(BF16), cache, dev(table),
                                           dev(np.array([n], np.int32)), dev(np.array([0, n], np.int32)), window=30,
                                           return_lse=True)
    torch.cuda.synchronize()
    rows = np.arange(70, 150)
    ref, rlse, _, tol, ltol = m.attend(q[:150], table, [150], np.array([0, 150]), 128 ** -0.5, True, 30)
    o, l = out.float().cpu().numpy()[rows], lse.cpu().numpy()[rows]
    assert np.all(np.isfinite(o)) and np.all(np.isfinite(l))
    t = tol[rows] + torch.finfo(BF16).eps / 2 * (np.abs(ref[rows]) + tol[rows])
    assert np.all(np.abs(o - ref[rows]) <= t) and np.all(np.abs(l - rlse[rows]) <= ltol[rows])


def test_attention_large_and_small_magnitudes(dq):
    """Queries, keys and values far from 1: one key takes nearly all the weight, or
    all keys weigh the same; values down to binary16's smallest scales."""
    rng = np.random.default_rng(15)
    lengths = [260]
    for kq, vv in ((2.0 ** 6, 1.0), (2.0 ** -20, 2.0 ** -15), (1.0, 2.0 ** 12), (1.0, 2.0 ** -22)):
        table, pages, starts = plan(rng, lengths, [1], 16)
        m = Model(pages, 16, 1, 128, 128, False)
        whole = np.array([0, 260], np.int32)
        m.write(values(rng, 260, 1, 128), values(rng, 260, 1, 128) * np.float32(vv), table, lengths, whole)
        q = rounded((rng.normal(size=(1, 4, 128)) * kq).astype(np.float32), BF16)
        check_attention(dq, m, table, lengths, None, q, BF16)


def test_attention_values_of_very_different_sizes(dq):
    """Scales of the values that grow and shrink by 2^20 along the sequence."""
    rng = np.random.default_rng(16)
    n = 700
    table, pages, starts = plan(rng, [n], [1], 16)
    m = Model(pages, 16, 1, 64, 64, False)
    grow = np.exp2(10 * np.sin(np.arange(n) / 40.0)).astype(np.float32)[:, None, None]
    m.write(values(rng, n, 1, 64), values(rng, n, 1, 64) * grow, table, [n], np.array([0, n], np.int32))
    q = rounded(rng.normal(size=(1, 3, 64)).astype(np.float32), F16)
    check_attention(dq, m, table, [n], None, q, F16)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_query_strides(dq, dtype):
    """Queries as a slice of a fused projection, at an odd address."""
    rng = np.random.default_rng(17)
    lengths, new, H, R, D = [50, 20], [6, 20], 2, 3, 80
    m, table, starts = filled(rng, H, D, 32, False, 16, lengths, new)
    q = rounded(rng.normal(size=(26, H * R, D)).astype(np.float32), dtype)
    cache = cache_of(dq, m)
    args = (cache, dev(table), dev(np.asarray(lengths, np.int32)), dev(starts))
    dense = dq.int4_cache_attention(torch.from_numpy(q).to(DEV).to(dtype), *args)
    for shape, pick in (((26, H * R + 2 * H, D), lambda t: t[:, :H * R]), ((H * R, 26, D), lambda t: t.transpose(0, 1))):
        buf = torch.zeros(int(np.prod(shape)) + 1, dtype=dtype, device=DEV)
        qs = pick(buf[1:].view(shape))
        qs.copy_(torch.from_numpy(q))
        assert torch.equal(dq.int4_cache_attention(qs, *args), dense)


# ---------------------------------------------------------------- together

def test_generation_with_the_cache(dq):
    """Prefill, then tokens one at a time, write before attend, against the model
    that sees the same writes; the last step replayed from a graph with other
    lengths and other tokens."""
    rng = np.random.default_rng(20)
    B, H, R, D, page = 3, 2, 4, 128, 16
    prompt, steps = [21, 1, 40], 5
    final = [p + steps for p in prompt]
    table, pages, starts = plan(rng, final, prompt, page)
    m = Model(pages, page, H, D, 64, True)
    cache = cache_of(dq, m)
    T = int(starts[-1])
    qkv = rounded(values(rng, T, H * R + 2 * H, D), BF16)
    x = torch.from_numpy(qkv).to(DEV).to(BF16)
    q, k, v = x[:, :H * R], x[:, H * R:H * R + H], x[:, H * R + H:]
    dq.int4_cache_write(cache, k, v, dev(table), dev(np.array(prompt, np.int32)), dev(starts))
    m.write(qkv[:, H * R:H * R + H], qkv[:, H * R + H:], table, prompt, starts)
    assert_same_bytes(cache, m)
    check_attention(dq, m, table, prompt, starts, qkv[:, :H * R], BF16, cache=cache)

    lens_d, x_d = dev(np.array(prompt, np.int32)), torch.zeros(B, H * R + 2 * H, D, dtype=BF16, device=DEV)
    table_d, out_d = dev(table), torch.zeros(B, H * R, D, dtype=BF16, device=DEV)
    ws = dq.cache_attention_workspace(cache, B, B, H * R)

    def step():
        dq.int4_cache_write(cache, x_d[:, H * R:H * R + H], x_d[:, H * R + H:], table_d, lens_d)
        dq.int4_cache_attention(x_d[:, :H * R], cache, table_d, lens_d, out=out_d, workspace=ws)

    graph, lens = None, list(prompt)
    for i in range(steps):
        new = rounded(values(rng, B, H * R + 2 * H, D), BF16)
        lens = [n + 1 for n in lens]
        lens_d.copy_(dev(np.array(lens, np.int32)))
        x_d.copy_(torch.from_numpy(new))
        if i == 2:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        if graph is not None:
            out_d.zero_()
            graph.replay()
        else:
            step()
        m.write(new[:, H * R:H * R + H], new[:, H * R + H:], table, lens, None)
        assert_same_bytes(cache, m)
        got = out_d.clone()
        want, _ = check_attention(dq, m, table, lens, None, new[:, :H * R], BF16, cache=cache)
        assert torch.equal(got, want), "captured or eager step differs from a direct call"


def test_two_streams_at_once(dq):
    rng = np.random.default_rng(21)
    cases = []
    for n in (900, 333):
        m, table, starts = filled(rng, 2, 64, 64, False, 16, [n], [1])
        q = rounded(rng.normal(size=(1, 4, 64)).astype(np.float32), F16)
        args = (torch.from_numpy(q).to(DEV).half(), cache_of(dq, m), dev(table), dev(np.array([n], np.int32)))
        cases.append((args, dq.int4_cache_attention(*args)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(10):
        for i, (args, _) in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i].append(dq.int4_cache_attention(*args))
    torch.cuda.synchronize()
    for i, (_, want) in enumerate(cases):
        assert all(torch.equal(g, want) for g in got[i])


def test_offsets_past_32_bits(dq):
    """Codes more than 2^32 bytes into the cache (the far pages of a 5 GB one)."""
    rng = np.random.default_rng(22)
    H, D, page = 1, 128, 1024
    m, table, starts = filled(rng, H, D, 128, False, 1024, [1500], [1500], spare=0)
    far = 2 ** 32 // (page * 64) + 5
    pages = far + 2
    cache = dq.Int4Cache.empty(pages, page, H, D, 128)
    for name, src in (("k_packed", m.packed["k"]), ("v_packed", m.packed["v"]), ("k_scales", m.scales["k"]),
                      ("v_scales", m.scales["v"])):
        getattr(cache, name)[far:far + 2] = dev(src)
    q = rounded(rng.normal(size=(3, 2, D)).astype(np.float32), BF16)
    check_attention(dq, m, table, [1500], np.array([0, 3], np.int32), q, BF16)
    near = dq.int4_cache_attention(dev(q).to(BF16), cache_of(dq, m), dev(table), dev(np.array([1500], np.int32)),
                                   dev(np.array([0, 3], np.int32)))
    t = dev(table + far)
    args = (t, dev(np.array([1500], np.int32)), dev(np.array([0, 3], np.int32)))
    assert torch.equal(dq.int4_cache_attention(dev(q).to(BF16), cache, *args), near)
    k = dev(values(rng, 3, H, D))
    dq.int4_cache_write(cache, k, -k, *args)
    m.write(k.cpu().numpy(), -k.cpu().numpy(), table, [1500], np.array([0, 3]))
    assert torch.equal(cache.k_packed[far:far + 2].cpu(), torch.from_numpy(m.packed["k"]))
    assert torch.equal(cache.v_packed[far:far + 2].cpu(), torch.from_numpy(m.packed["v"]))
    got = dq.int4_cache_read(cache, *args, rows=3, dtype=F32)
    assert np.array_equal(got[0].cpu().numpy(), m.read(3, table, [1500], np.array([0, 3]))[0])
