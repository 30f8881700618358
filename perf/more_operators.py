"""Cases and plain forms of the operators of a serving step over the 4-bit
key/value cache: pages for new tokens (int4_cache_release, int4_cache_extend),
norms, rotation and write in one pass (int4_cache_append), attention with a
window and first tokens that stay visible, and attention for a batch that
shares its first tokens (int4_cache_attention, sinks= and shared=).

A case is one of four operators, "op":
  pages   finished sequences give their pages back, the others get pages for
          their new tokens: lengths, row offsets, the slot of each row
  append  queries and keys are normalised for each head and rotated, queries are
          returned, keys and values quantised into the cache; the values that the
          written codes stand for are read back
  sinks   rows of queries see the last ``window`` keys and the first ``sinks``
  shared  all sequences begin with the same ``shared`` tokens, on the same pages

Sizes: ``batch`` sequences, lengths between ``len_lo`` and ``len_hi`` (cached
tokens, the new ones included, the shared ones not), new rows a sequence between
``new_lo`` and ``new_hi``; ``heads`` key/value heads of ``head_dim`` channels,
``ratio`` query heads for each; ``page`` tokens a page; ``group`` channels a
scale; ``affine`` codes with zero points or symmetric ones; ``rotary`` channels
that are rotated (0: none), ``interleaved`` pairs or halves; ``norm``.

The cache's layout is that of include/int4dq_cache.h (C = 2, 3, 4, 6 or 8 blocks
of 32 channels that hold head_dim, DB = 16 C):
  k_packed [pages, heads, page, DB]: a token's row; channel d = 32 i + 8 a + e is nibble e % 2 of
           byte 4 C a + 4 i + e // 2
  v_packed [pages, heads, page / 16, DB, 16]: 16 tokens; channel d of token t is nibble d % 2 of byte [d // 2, t % 16]
  scales   [pages, heads, page / 16, G, 16] binary16, zero points alike in bytes
"""
import math

import torch

own = False

DTYPES = {"float16": torch.float16, "bfloat16": torch.bfloat16, "float32": torch.float32}
EPS = 1e-6


def _case(name, op, batch, len_lo, len_hi, new_lo, new_hi, page, heads=8, ratio=4, head_dim=128, group=128,
          affine=False, dtype="bfloat16", **more):
    return {"name": name, "op": op, "batch": batch, "len_lo": len_lo, "len_hi": len_hi, "new_lo": new_lo,
            "new_hi": new_hi, "page": page, "heads": heads, "ratio": ratio, "head_dim": head_dim, "group": group,
            "affine": affine, "dtype": dtype, **more}


def listed():
    return [
        # one generated token for each of a serving batch, a few of which have ended: latency
        _case("pages_step", "pages", 128, 5, 4000, 1, 1, 64, done=9),
        # a prefill step: prompts of uneven lengths, some of them continued
        _case("pages_prompts", "pages", 48, 40, 9000, 30, 4000, 16, done=2),
        # one generated token of one sequence: latency
        _case("append_one", "append", 1, 700, 700, 1, 1, 64, rotary=128, interleaved=False, norm=True),
        # one token for each of a batch of sequences, affine codes, a part of the channels rotated in pairs
        _case("append_batch", "append", 128, 5, 4000, 1, 1, 64, group=64, affine=True, dtype="float16", rotary=64,
              interleaved=True, norm=True),
        # prompts of uneven lengths, some onto cached prefixes, as a prefill step writes them
        _case("append_prompts", "append", 12, 900, 6000, 300, 4100, 64, rotary=128, interleaved=False, norm=True),
        # token generation in long conversations that keep a window and their first tokens
        _case("sinks_decode", "sinks", 32, 500, 16001, 1, 1, 64, window=2048, sinks=4),
        # one long conversation, small groups with zero points
        _case("sinks_one", "sinks", 1, 60001, 60001, 1, 1, 256, group=32, affine=True, dtype="float16", window=8192,
              sinks=64),
        # chunks of long prompts
        _case("sinks_prompts", "sinks", 4, 3000, 9001, 257, 1024, 64, heads=4, ratio=6, head_dim=96, group=96,
              dtype="float16", window=1500, sinks=100),
        # a few answers to one short system prompt: latency
        _case("shared_few", "shared", 6, 20, 300, 1, 1, 64, shared=1984),
        # a serving batch whose requests share a long document
        _case("shared_decode", "shared", 64, 10, 1500, 1, 1, 64, group=64, shared=32768),
        # as many key heads as query heads, 768 = 12 x 64 channels, a large batch
        _case("shared_small_model", "shared", 200, 1, 200, 1, 1, 16, heads=12, ratio=1, head_dim=64, group=64,
              dtype="float16", shared=4000),
        # questions of some length about one document, as a prefill step computes them
        _case("shared_questions", "shared", 16, 30, 400, 30, 250, 64, shared=20011),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["pages", "append", "append", "sinks", "sinks", "shared", "shared"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "pages":
        batch = spread(1, 1000)
        hi = spread(4, 9000)
        lo = max(1, hi // rng.choice([1, 3, 10]))
        new = (1, 1) if rng.random() < 0.5 else (max(1, lo // 2), lo)
        new = (min(new[0], max(1, 60000 // batch)), min(new[1], max(1, 60000 // batch)))
        return _case("", op, batch, lo, hi, *new, page, done=rng.choice([0, 1, batch // 5]))
    head_dim = rng.choice([64, 72, 80, 96, 128, 128, 160, 192, 256])
    group = rng.choice([32, 64, 128])
    heads = rng.choice([1, 2, 4, 5, 8, 8, 12])
    ratio = rng.choice([1, 2, 4, 5, 7, 8])
    affine = rng.random() < 0.4
    batch = spread(1, 128)
    if op == "append":
        dtype = rng.choice(["float16", "bfloat16", "float32"])
        most = max(8, int(2.0e7 / (batch * heads * (ratio + 2) * head_dim)))
        hi = spread(4, most)
        lo = max(1, hi // rng.choice([1, 2, 5]))
        new = (max(1, lo // 2), lo) if rng.random() < 0.6 else (1, 1)
        rotary = rng.choice([0, head_dim, head_dim, head_dim // 2])
        return _case("", op, batch, lo, hi, *new, page, heads, ratio, head_dim, group, affine, dtype, rotary=rotary,
                     interleaved=rng.random() < 0.4, norm=rng.random() < 0.7)
    dtype = rng.choice(["float16", "bfloat16"])
    kind = rng.choice(["decode", "decode", "few", "prompt"])
    if kind == "prompt":
        batch = spread(1, 6)
        hi = spread(40, max(64, int(math.sqrt(4.0e9 / (batch * heads * ratio * head_dim)))))
        lo = max(1, hi // 2)
        new = (max(1, lo // 3), lo)
    else:
        hi = spread(8, min(30000, max(16, int(4e7 / (batch * heads * head_dim)))))
        lo = max(1, hi // rng.choice([1, 3, 10]))
        new = (1, 1) if kind == "decode" else (1, min(lo, 8))
    if op == "sinks":
        return _case("", op, batch, lo, hi, *new, page, heads, ratio, head_dim, group, affine, dtype,
                     window=rng.choice([1, 128, 1000, 2048]), sinks=rng.choice([1, 4, 16, 64, 129]))
    lo, hi = min(lo, 1500), min(hi, 3000)
    new = (min(new[0], lo), min(new[1], lo))
    rows = batch * (new[0] + new[1]) * heads * ratio * head_dim / 2
    return _case("", op, batch, lo, hi, *new, page, heads, ratio, head_dim, group, affine, dtype,
                 shared=spread(100, max(200, min(33000, int(8.0e9 / rows)))))


def _between(lo, hi, n, step):
    """n whole numbers spread over lo .. hi, the largest among them, the same for the same arguments."""
    return [hi - (i * step) % (hi - lo + 1) for i in range(n)]


def _sizes(case):
    """Cached tokens and new rows of each sequence, the shared ones not counted."""
    lens = _between(case["len_lo"], case["len_hi"], case["batch"], 2654435761 % (case["len_hi"] - case["len_lo"] + 1) or 1)
    new = _between(case["new_lo"], case["new_hi"], case["batch"], 7 * (case["new_hi"] - case["new_lo"]) // 13 or 1)
    return lens, [min(n, m) for n, m in zip(new, lens)]


def _done(case):
    """Which sequences have ended."""
    return [i * case["done"] // case["batch"] != (i + 1) * case["done"] // case["batch"] for i in range(case["batch"])]


def _blocks(head_dim):
    return next(c for c in (2, 3, 4, 6, 8) if 32 * c >= head_dim)


def _groups(case):
    return -(-case["head_dim"] // case["group"])


def work(case):
    lens, new = _sizes(case)
    S = case["page"]
    if case["op"] == "pages":
        done = _done(case)
        rows = sum(m for m, d in zip(new, done) if not d)
        given = sum(-(-(n - m) // S) for n, m, d in zip(lens, new, done) if d)
        taken = sum(-(-n // S) - -(-(n - m) // S) for n, m, d in zip(lens, new, done) if not d)
        return {"bytes": 8 * rows + 8 * (given + taken) + 21 * case["batch"] + 20, "flops": 4.0 * rows}
    H, D, G, R = case["heads"], case["head_dim"], _groups(case), case["ratio"]
    held = 2 * (D / 2 + G * (3 if case["affine"] else 2)) * H       # bytes of a cached token, keys and values
    value = 4 if case["dtype"] == "float32" else 2
    plan = 4 * (2 * case["batch"] + 1)
    rows = sum(new)
    if case["op"] == "append":
        # read the new rows, write queries and codes; read the codes back, write the values
        return {"bytes": rows * (2 * H * R * D * value + 2 * (held + 2 * H * D * value) + 4 * case["rotary"]) + plan,
                "flops": rows * H * D * (12.0 + 6.0 * (R + 1))}
    pairs, seen = 0, case.get("shared", 0)
    for n, m in zip(lens, new):
        first = n - m                                # positions first .. n - 1
        if case["op"] == "shared":
            pairs += m * (case["shared"] + first) + m * (m + 1) // 2
            seen += n
        else:
            w, s = case["window"], case["sinks"]
            pairs += sum(min(p + 1, w + min(s, max(0, p + 1 - w))) for p in range(first, n))
            seen += min(n, w + m - 1 + min(s, max(0, n - w)))
    return {"bytes": seen * held + rows * H * R * (2 * D * value + 4) + plan, "flops": 4.0 * D * R * H * pairs}


# ------------------------------------------------------------ inputs

def _quantise(x, group, affine):
    """x [..., D] float32 -> nibbles uint8 [..., D], scales float16 [..., G], zero points uint8 [..., G] or None."""
    D = x.shape[-1]
    G = -(-D // group)
    wide = torch.nn.functional.pad(x, (0, G * group - D)).reshape(*x.shape[:-1], G, group)
    if affine:
        lo, hi = wide.amin(-1).clamp(max=0.0), wide.amax(-1).clamp(min=0.0)
        scale = ((hi - lo) / 15.0).half()
        s = scale.float()
        zero = torch.where(s > 0, torch.round(-lo / s).clamp(0, 15), torch.zeros_like(s))
        # the sum of quotient and zero point is exact in 64 bits
        u = torch.round((wide / s[..., None]).double() + zero[..., None].double()).clamp(0, 15)
        u = torch.where(s[..., None] > 0, u, torch.zeros_like(u)).to(torch.uint8)
        return u.reshape(*x.shape[:-1], G * group)[..., :D], scale, zero.to(torch.uint8)
    scale = (wide.abs().amax(-1) / 7.0).half()
    s = scale.float()[..., None]
    q = torch.where(s > 0, torch.round(wide / s).clamp(-8, 7), torch.zeros_like(wide)).to(torch.int8)
    return (q & 15).to(torch.uint8).reshape(*x.shape[:-1], G * group)[..., :D], scale, None


def _pairs(nibbles, blocks):
    wide = torch.nn.functional.pad(nibbles, (0, 32 * blocks - nibbles.shape[-1]))
    return wide[..., 0::2] | (wide[..., 1::2] << 4)          # [..., DB] bytes, channels in order


def _key_rows(nibbles, blocks):
    b = _pairs(nibbles, blocks)
    return b.reshape(*b.shape[:-1], blocks, 4, 4).transpose(-3, -2).reshape(b.shape)


def _sixteens(t):
    """[..., page, n] -> [..., page / 16, n, 16]."""
    return t.reshape(*t.shape[:-2], t.shape[-2] // 16, 16, t.shape[-1]).transpose(-1, -2).contiguous()


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    lens, new = _sizes(case)
    B, S = case["batch"], case["page"]
    if case["op"] == "pages":
        done = _done(case)
        new = [0 if d else m for m, d in zip(new, done)]
        old = [n - m for n, m in zip(lens, new)]
        held = [-(-n // S) for n in old]
        need = sum(-(-n // S) for n in lens) + 40
        most = max(-(-n // S) for n in lens) + 2
        order = torch.randperm(sum(held) + need, generator=g, device=dev).to(torch.int32)
        table = torch.full((B, most), -1, dtype=torch.int32, device=dev)
        at = 0
        for b, n in enumerate(held):
            table[b, :n] = order[at:at + n]
            at += n
        free = torch.full_like(order, -1)
        free[:need] = order[at:]
        return {"case": case, "page_table": table, "free": free, "rows": sum(new),
                "count": torch.tensor([need, 0], dtype=torch.int32, device=dev),
                "lengths": torch.tensor(old, dtype=torch.int32, device=dev),
                "new": torch.tensor(new, dtype=torch.int32, device=dev),
                "done": torch.tensor(done, dtype=torch.bool, device=dev)}
    H, D, R = case["heads"], case["head_dim"], case["ratio"]
    C, G, dtype = _blocks(D), _groups(case), DTYPES[case["dtype"]]
    shared = case.get("shared", 0)
    common = -(-shared // S)                                 # pages that all sequences have
    lens = [common * S + n for n in lens]
    counts = [-(-n // S) for n in lens]
    pages = sum(c - common for c in counts) + common + 3     # a few that no sequence owns
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, max(counts)), -1, dtype=torch.int32, device=dev)
    table[:, :common] = order[:common]
    at = common
    for b, c in enumerate(counts):
        table[b, common:c] = order[at:at + c - common]
        at += c - common
    starts = torch.tensor([0] + new, dtype=torch.int64).cumsum(0).to(torch.int32).to(dev)
    state = {"case": case, "page_table": table, "starts": None if set(new) == {1} else starts,
             "lengths": torch.tensor(lens, dtype=torch.int32, device=dev), "rows": sum(new), "most": max(new),
             "shared": torch.tensor([shared], dtype=torch.int32, device=dev) if shared else None}

    def values(*shape):
        # keys and values of a trained model: a few channels are much larger than the rest
        channel = torch.exp(0.6 * torch.randn(H, D, generator=g, device=dev))
        return torch.randn(*shape, H, D, generator=g, device=dev) * channel

    if case["op"] == "append":
        state["k_packed"] = torch.zeros(pages, H, S, 16 * C, dtype=torch.uint8, device=dev)
        state["v_packed"] = torch.zeros(pages, H, S // 16, 16 * C, 16, dtype=torch.uint8, device=dev)
        for side in ("k", "v"):
            state[side + "_scales"] = torch.zeros(pages, H, S // 16, G, 16, dtype=torch.float16, device=dev)
            state[side + "_zeros"] = torch.zeros(pages, H, S // 16, G, 16, dtype=torch.uint8, device=dev) if case["affine"] else None
        # queries, keys and values are slices of one projection's output
        q = torch.randn(sum(new), H * R, D, generator=g, device=dev) * torch.exp(0.6 * torch.randn(D, generator=g, device=dev))
        fused = torch.cat([q, values(sum(new)), values(sum(new))], 1).to(dtype)
        state["q"], state["k"], state["v"] = fused[:, :H * R], fused[:, H * R:H * R + H], fused[:, H * R + H:]
        weight = 1.0 + 0.3 * torch.randn(2, D, generator=g, device=dev)
        state["q_norm"], state["k_norm"] = weight.unbind(0) if case["norm"] else (None, None)
        state["rope"] = None
        if case["rotary"]:
            half = case["rotary"] // 2
            angle = torch.outer(torch.arange(max(lens) + 100, dtype=torch.float64, device=dev),
                                500000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half))
            state["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        return state
    for side in ("k", "v"):
        n, s, z = _quantise(values(pages, S).transpose(1, 2).contiguous(), case["group"], case["affine"])
        state[side + "_packed"] = _key_rows(n, C) if side == "k" else _sixteens(_pairs(n, C))
        state[side + "_scales"] = _sixteens(s)
        state[side + "_zeros"] = None if z is None else _sixteens(z)
    state["q"] = torch.randn(sum(new), H * R, D, generator=g, device=dev).to(dtype)
    return state


# ------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    import dequantizing_gemm_amd as dq
    case = state["case"]
    if case["op"] == "pages":
        table, free, S = state["page_table"], state["free"], case["page"]
        lengths, count = dq.int4_cache_release(table, state["lengths"], free, state["count"], S, state["done"])
        lengths, starts, slots, count = dq.int4_cache_extend(table, lengths, free, count, S, state["new"], rows=state["rows"])
        return {"page_table": table, "lengths": lengths, "starts": starts, "slots": slots, "count": count}
    if "cache" not in state:
        state["cache"] = dq.Int4Cache(state["k_packed"], state["k_scales"], state["v_packed"], state["v_scales"],
                                      case["head_dim"], case["group"], state["k_zeros"], state["v_zeros"])
    cache, plan = state["cache"], (state["page_table"], state["lengths"], state["starts"])
    if case["op"] == "append":
        q = dq.int4_cache_append(cache, state["q"], state["k"], state["v"], *plan, q_norm=state["q_norm"],
                                 k_norm=state["k_norm"], eps=EPS, rope=state["rope"], interleaved=case["interleaved"])
        k, v = dq.int4_cache_read(cache, *plan, rows=state["rows"], dtype=DTYPES[case["dtype"]])
        return q, k, v
    if case["op"] == "sinks":
        return dq.int4_cache_attention(state["q"], cache, *plan, window=case["window"], sinks=case["sinks"], return_lse=True)
    return dq.int4_cache_attention(state["q"], cache, *plan, shared=state["shared"], return_lse=True)


def _run_plain(state):
    case = state["case"]
    if case["op"] == "pages":
        return _pages_plain(state)
    return _append_plain(state) if case["op"] == "append" else _attend_plain(state)


def _pages_plain(state):
    S, table, free = state["case"]["page"], state["page_table"], state["free"]
    B, most = table.shape
    lens, new, count = state["lengths"].long(), state["new"].long(), state["count"][0].long()
    done = state["done"]
    index = torch.arange(most, device=table.device)
    # pages of ended sequences go back, in the order of the table
    held = ((lens + S - 1) // S).clamp(max=most)
    back = ((index < held[:, None]) & done[:, None]).flatten()
    place = torch.where(back, count + back.cumsum(0) - 1, free.shape[0])
    room = torch.cat([free, free[:1]])
    room[place] = table.flatten()
    free.copy_(room[:-1])
    count = count + back.sum()
    lens = torch.where(done, 0, lens)
    # pages for the new tokens
    held = ((lens + S - 1) // S).clamp(max=most)
    need = ((lens + new + S - 1) // S).clamp(max=most) - held
    before = need.cumsum(0) - need
    fresh = (index >= held[:, None]) & (index < (held + need)[:, None])
    at = count - 1 - before[:, None] - (index - held[:, None])
    pages = torch.where(at >= 0, free[at.clamp(0, free.shape[0] - 1)], -1)
    table.copy_(torch.where(fresh, pages, table))
    lens = lens + new
    starts = torch.cat([new.new_zeros(1), new.cumsum(0)])
    seq = torch.repeat_interleave(torch.arange(B, device=lens.device), new, output_size=state["rows"])
    pos = lens[seq] - starts[1:][seq] + torch.arange(state["rows"], device=lens.device)
    page = table[seq, (pos // S).clamp(max=most - 1)].long()
    slots = torch.where((page >= 0) & (pos // S < most), page * S + pos % S, -1)
    left = count - need.sum()
    return {"page_table": table, "lengths": lens.int(), "starts": starts.int(), "slots": slots,
            "count": torch.stack([left.clamp(min=0), (-left).clamp(min=0)]).int()}


def _positions(state):
    """The sequence and the position of each row."""
    lens = state["lengths"].long()
    B = lens.shape[0]
    if state["starts"] is None:
        return torch.arange(B, device=lens.device), lens - 1
    starts = state["starts"].long()
    seq = torch.repeat_interleave(torch.arange(B, device=lens.device), starts[1:] - starts[:-1], output_size=state["rows"])
    return seq, lens[seq] - starts[1:][seq] + torch.arange(state["rows"], device=lens.device)


def _values(nibbles, scale, zero, group):
    """What nibbles [..., D] stand for, in 32 bits: scales and zero points [..., G]."""
    D = nibbles.shape[-1]
    s = scale.float().repeat_interleave(group, -1)[..., :D]
    if zero is None:
        return ((nibbles ^ 8).float() - 8.0) * s
    return (nibbles.float() - zero.float().repeat_interleave(group, -1)[..., :D]) * s


def _nibbles(rows, D):
    return torch.stack([rows & 15, rows >> 4], -1).flatten(-2)[..., :D]


def _key_bytes(rows, blocks):
    """Bytes of key rows [..., DB], channels in order."""
    return rows.reshape(*rows.shape[:-1], 4, blocks, 4).transpose(-3, -2).reshape(rows.shape)


def _normed_rotated(x, weight, rope, interleaved):
    """x [rows, heads, D] float32. The codes of a key next to a border go by the last bit of this: the mean is taken
    in 64 bits, and then each product and sum is rounded once."""
    if weight is not None:
        r = (1.0 / torch.sqrt(x.double().square().mean(-1, keepdim=True) + EPS)).float()
        x = x * r * weight
    if rope is None:
        return x
    half = rope.shape[1] // 2
    c, s = rope[:, None, :half], rope[:, None, half:]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _append_plain(state):
    case = state["case"]
    D, S, C, group = case["head_dim"], case["page"], _blocks(case["head_dim"]), case["group"]
    dtype = DTYPES[case["dtype"]]
    seq, pos = _positions(state)
    page = state["page_table"].long()[seq, pos // S]
    slot = pos % S
    six, lane = slot // 16, slot % 16
    rope = None if state["rope"] is None else state["rope"][pos]
    q = _normed_rotated(state["q"].float(), state["q_norm"], rope, case["interleaved"])
    out = [q.to(dtype)]
    for side in ("k", "v"):
        x = state[side].float()
        if side == "k":
            x = _normed_rotated(x, state["k_norm"], rope, case["interleaved"])
        n, s, z = _quantise(x, group, case["affine"])
        if side == "k":
            state["k_packed"][page, :, slot] = _key_rows(n, C)
            b = _key_bytes(state["k_packed"][page, :, slot], C)
        else:
            state["v_packed"][page, :, six, :, lane] = _pairs(n, C)
            b = state["v_packed"][page, :, six, :, lane]
        state[side + "_scales"][page, :, six, :, lane] = s
        if z is not None:
            state[side + "_zeros"][page, :, six, :, lane] = z
        z = state[side + "_zeros"]
        out.append(_values(_nibbles(b, D), state[side + "_scales"][page, :, six, :, lane],
                           None if z is None else z[page, :, six, :, lane], group).to(dtype))
    return tuple(out)


def _tokens(t):
    """Gathered pages [B, n, H, page / 16, m, 16] -> [B, H, tokens, m]."""
    t = t.transpose(-1, -2).transpose(1, 2)
    return t.reshape(t.shape[0], t.shape[1], -1, t.shape[-1])


def _held(state, table):
    """Keys and values [B, H, tokens, D] in 32 bits of the pages of a table [B, n]."""
    case = state["case"]
    D, C, H, group = case["head_dim"], _blocks(case["head_dim"]), case["heads"], case["group"]
    rows = state["k_packed"][table].transpose(1, 2).reshape(table.shape[0], H, -1, 16 * C)

    def of(side, rows):
        z = state[side + "_zeros"]
        return _values(_nibbles(rows, D), _tokens(state[side + "_scales"][table]), None if z is None else _tokens(z[table]), group)

    return of("k", _key_bytes(rows, C)), of("v", _tokens(state["v_packed"][table]))


def _attend_plain(state):
    case = state["case"]
    H, R, D, S = case["heads"], case["ratio"], case["head_dim"], case["page"]
    lens, table = state["lengths"].long(), state["page_table"].long().clamp(min=0)
    B, dev, q, most = lens.shape[0], lens.device, state["q"], state["most"]
    starts = torch.arange(B + 1, device=dev) if state["starts"] is None else state["starts"].long()
    new = starts[1:] - starts[:-1]
    common = -(-case.get("shared", 0) // S)
    # rows of the batch, padded to the longest: [B, H, most * R, D]
    at = starts[:-1, None] + torch.arange(most, device=dev)
    there = torch.arange(most, device=dev) < new[:, None]
    qs = q.float()[at.clamp(max=q.shape[0] - 1)].reshape(B, most, H, R, D).transpose(1, 2).reshape(B, H, most * R, D)
    pos = (lens - new)[:, None] + torch.arange(most, device=dev)               # [B, most]
    k, v = _held(state, table[:, common:])
    a = torch.matmul(qs, k.transpose(-1, -2).contiguous())
    if common:
        # the shared pages once, for the rows of all sequences side by side
        k0, v0 = _held(state, table[:1, :common])
        flat = qs.transpose(0, 1).reshape(H, B * most * R, D)
        a0 = torch.matmul(flat, k0[0].transpose(-1, -2).contiguous()).reshape(H, B, most * R, -1).transpose(0, 1)
        a = torch.cat([a0, a], -1)
    key = torch.arange(a.shape[-1], device=dev)
    seen = (key <= pos[..., None]) & (key < lens[:, None, None])
    if case["op"] == "sinks":
        seen &= (key > pos[..., None] - case["window"]) | (key < case["sinks"])
    a = (a * (1.0 / math.sqrt(D))).reshape(B, H, most, R, -1).masked_fill_(~seen[:, None, :, None], -math.inf)
    top = a.amax(-1, keepdim=True)
    p = torch.exp(a - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    p = p.reshape(B, H, most * R, -1)
    o = torch.matmul(p[..., common * S:], v)
    if common:
        p0 = p[..., :common * S].transpose(0, 1).reshape(H, B * most * R, -1)
        o = o + torch.matmul(p0, v0[0]).reshape(H, B, most * R, D).transpose(0, 1)
    o = o.reshape(B, H, most, R, D) / total.clamp(min=1e-37)
    lse = (top + torch.log(total)).squeeze(-1)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, most, H * R, D)[there]
    lse = lse.permute(0, 2, 1, 3).reshape(B, most, H * R)[there]
    return o.to(q.dtype), lse


# ------------------------------------------------------------ from the definition, in 64 bits

def _exact_pages(case, state):
    S, table = case["page"], state["page_table"].tolist()
    free, left = state["free"].tolist(), state["count"].tolist()[0]
    stack, lens, new = free[:left], state["lengths"].tolist(), state["new"].tolist()
    for b, ended in enumerate(_done(case)):
        if ended:
            stack += table[b][:-(-lens[b] // S)]
            lens[b] = 0
    starts, slots, lacking = [0], [], 0
    for b, m in enumerate(new):
        for p in range(lens[b], lens[b] + m):
            if p // S < len(table[b]):
                if p % S == 0:
                    lacking += not stack
                    table[b][p // S] = stack.pop() if stack else -1
                slots.append(table[b][p // S] * S + p % S if table[b][p // S] >= 0 else -1)
            else:
                slots.append(-1)
        lens[b] += m
        starts.append(starts[-1] + m)
    return {"page_table": torch.tensor(table, dtype=torch.int32), "lengths": torch.tensor(lens, dtype=torch.int32),
            "starts": torch.tensor(starts, dtype=torch.int32), "slots": torch.tensor(slots, dtype=torch.int64),
            "count": torch.tensor([len(stack), lacking], dtype=torch.int32)}


def _exact_append(case, state):
    D, group, affine = case["head_dim"], case["group"], case["affine"]
    lens, new = _sizes(case)
    pos = torch.tensor([p for n, m in zip(lens, new) for p in range(n - m, n)], device=state["q"].device)
    x = {n: state[n].double() for n in "qkv"}
    for n in "qk":
        w = state[n + "_norm"]
        if w is not None:
            x[n] = x[n] / torch.sqrt((x[n] ** 2).sum(-1, keepdim=True) / D + EPS) * w.double()
        if state["rope"] is not None:
            half = case["rotary"] // 2
            turn = torch.complex(*state["rope"][pos].double().split(half, 1))[:, None]
            i = torch.arange(half, device=pos.device)
            first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
            z = torch.complex(x[n][..., first], x[n][..., second]) * turn
            x[n] = x[n].clone()
            x[n][..., first], x[n][..., second] = z.real, z.imag
    out = [x["q"]]
    for n in "kv":
        y = torch.empty_like(x[n], memory_format=torch.contiguous_format)
        for i in range(_groups(case)):
            part = x[n][..., i * group:(i + 1) * group].float().double()        # keys are rounded to binary32 first
            if affine:
                lo, hi = part.amin(-1, True).clamp(max=0), part.amax(-1, True).clamp(min=0)
                # the scale is the binary16 of a binary32 quotient
                s = ((hi - lo).float().double() / 15).float().half().double()
                z = torch.round((-lo / s).float().double()).clamp(0, 15)
                c = torch.round((part / s).float().double() + z).clamp(0, 15) - z
            else:
                s = (part.abs().amax(-1, True) / 7).float().half().double()
                c = torch.round((part / s).float().double()).clamp(-8, 7)
            y[..., i * group:(i + 1) * group] = torch.where(s > 0, c * s, torch.zeros_like(c))
        out.append(y)
    return tuple(out)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "pages":
        return _exact_pages(case, state)
    if case["op"] == "append":
        return _exact_append(case, state)
    _, new = _sizes(case)
    lens = state["lengths"].tolist()
    H, D, S, R, group = case["heads"], case["head_dim"], case["page"], case["ratio"], case["group"]
    C, affine = _blocks(D), case["affine"]
    dev = state["lengths"].device
    d = torch.arange(D, device=dev)
    i, a, e = d // 32, d % 32 // 8, d % 8

    def cached(side, b, p):
        """[H, n, D]: what sequence b holds at positions p."""
        page, slot = state["page_table"][b].long()[p // S][:, None], (p % S)[:, None]
        if side == "k":
            byte, odd = state["k_packed"].permute(0, 2, 3, 1)[page, slot, 4 * C * a + 4 * i + e // 2], e % 2
        else:
            byte, odd = state["v_packed"].permute(0, 2, 3, 4, 1)[page, slot // 16, d // 2, slot % 16], d % 2
        c = (byte.long() >> (4 * odd)[:, None]) % 16                   # [tokens, D, H]
        s = state[side + "_scales"].permute(0, 2, 3, 4, 1)[page, slot // 16, d // group, slot % 16].double()
        if affine:
            c = c - state[side + "_zeros"].permute(0, 2, 3, 4, 1)[page, slot // 16, d // group, slot % 16].long()
        else:
            c = torch.where(c > 7, c - 16, c)
        return (c.double() * s).permute(2, 0, 1)

    head = torch.arange(case.get("shared", 0), device=dev)
    first = {side: cached(side, 0, head) for side in "kv"} if len(head) else None
    outs, lses, at = [], [], 0
    for b, (n, m) in enumerate(zip(lens, new)):
        key = torch.arange(n, device=dev)
        if case["op"] == "sinks":                    # those that some row sees
            key = key[(key > n - m - case["window"]) | (key < case["sinks"])]
        k, v = (cached(side, b, key[len(head):]) for side in "kv")
        if first:
            k, v = torch.cat([first["k"], k], 1), torch.cat([first["v"], v], 1)
        q = state["q"][at:at + m].double().reshape(m, H, R, D).permute(1, 2, 0, 3).reshape(H, R * m, D)
        at += m
        s = torch.bmm(q, k.transpose(1, 2).contiguous()).reshape(H, R, m, len(key)) / math.sqrt(D)
        pos = torch.arange(n - m, n, device=dev)[:, None]
        hide = key > pos
        if case["op"] == "sinks":
            hide = hide | ((key <= pos - case["window"]) & (key >= case["sinks"]))
        s = s.masked_fill(hide, -math.inf)
        lses.append(torch.logsumexp(s, -1).permute(2, 0, 1).reshape(m, H * R))
        o = torch.bmm(torch.softmax(s, -1).reshape(H, R * m, len(key)), v)
        outs.append(o.reshape(H, R, m, D).permute(2, 0, 1, 3).reshape(m, H * R, D))
    return torch.cat(outs), torch.cat(lses)
