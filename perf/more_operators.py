"""What is timed of the 8-bit KV cache and its rotary tables: cos/sin rows for positions, storing new K/V
rows in 8 bits (rotated on the way, or as they are), loading rows back, and decode attention.

The cache format.  `block` consecutive rows of the pool are a block of tokens.  A block has, for each
head and for K and V apart, one exponent e (a byte, e + 127), and every channel of every row an element c
in e4m3; a channel stands for c * 2**e.  The exponent that values need is the smallest e, from -120 to
119, with max |x| <= 448 * 2**e.  A store whose first row in a block is the block's first gives it the
exponent that its new rows need.  A store that goes on in a block gives it the larger of that and the
block's exponent so far, and rounds the older rows again where it grew.  Elements are rounded to
nearest, ties to even.

Rotary positions.  The first `rotary` channels of a q or k head are rotated in pairs, channel j with
channel j + rotary/2, or 2j with 2j+1 where interleaved, by the angle p * theta_j; row p of the table is
[cos | sin].  The frequencies are base**(-2j/rotary), scaled for long contexts in one of four ways.

Every case is one pass through one operator, with `run` in two forms: plain torch operations (own is
False) and the library's calls (own is True).
"""
import math
import random

import numpy as np
import torch

own = False

TOP = 448.0  # the largest e4m3 element
LOWEST, HIGHEST = -120, 119  # exponents


# --------------------------------------------------------------------------- #
# cases
# --------------------------------------------------------------------------- #
def listed():
    return [
        # the rows of one chunked-prefill step's tokens, wherever they are in a long context
        dict(name="table-step", op="table", rotary=64, count=2048, spread=1_000_000, base=10000.0, kind="linear",
             factor=8.0, origin=8192),
        # the whole table of a context of 128k, made when an engine starts
        dict(name="table-128k", op="table", rotary=128, count=131072, spread=0, base=10000.0, kind="yarn", factor=32.0,
             origin=4096),
        # one new token of each of 64 requests, which goes on in a block of 16: latency
        dict(name="store-step", op="store", heads=8, group=4, dim=128, batch=64, lo=700, hi=4096, new_lo=1, new_hi=1,
             rotary=128, pairs="half", block=16, page=16),
        # a chunked-prefill batch of about 8k new tokens behind cached prefixes of any length
        dict(name="store-chunk", op="store", heads=8, group=4, dim=128, batch=13, lo=1, hi=3000, new_lo=256,
             new_hi=1024, rotary=128, pairs="half", block=16, page=64),
        # rows that are rotated already, every row a block of its own: a pool of single-row pages
        dict(name="store-rows", op="store", heads=8, group=0, dim=128, batch=40, lo=0, hi=0, new_lo=1, new_hi=2047,
             rotary=0, pairs="half", block=1, page=1),
        # many prompts at once, ragged, head_dim 64 of which half is rotated, neighbours in pairs
        dict(name="store-prompts", op="store", heads=5, group=3, dim=64, batch=96, lo=0, hi=0, new_lo=1, new_hi=2777,
             rotary=32, pairs="interleaved", block=64, page=64),
        # a chunk's cached prefixes read back for the prefill attention, one request without any
        dict(name="load-chunk", op="load", heads=8, dim=128, batch=13, lo=2048, hi=3056, log=False, empty=1, block=1,
             page=1),
        # long prefixes read back, 64-row pages
        dict(name="load-long", op="load", heads=8, dim=128, batch=16, lo=8193, hi=32769, log=False, empty=0, block=64,
             page=64),
        # one token for each of four short chats on a small model: the smallest decode call
        dict(name="decode-tiny", op="decode", heads=2, group=4, dim=64, batch=4, lo=17, hi=129, log=False, empty=0,
             block=16, page=16),
        # an ordinary decode step: 64 requests of 512 to 4096 cached tokens, single-row pages
        dict(name="decode-b64", op="decode", heads=8, group=2, dim=128, batch=64, lo=513, hi=4097, log=False, empty=0,
             block=1, page=1),
        # a full batch, 1k to 8k tokens each, with 56 empty slots behind the live requests
        dict(name="decode-b256", op="decode", heads=8, group=4, dim=128, batch=256, lo=1025, hi=8193, log=True,
             empty=56, block=16, page=16),
        # a few long contexts in 64-row pages, eight query heads to a KV head
        dict(name="decode-long", op="decode", heads=8, group=8, dim=128, batch=6, lo=32769, hi=131073, log=False,
             empty=0, block=64, page=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(("decode", "decode", "store", "store", "load", "table"))
    if op == "table":
        kind = rng.choice(("plain", "linear", "ntk", "bands", "yarn"))
        return dict(op=op, rotary=rng.choice((16, 32, 64, 96, 128, 128)), count=_log_int(rng, 1, 120_000),
                    spread=rng.choice((0, _log_int(rng, 1000, 4_000_000))), base=rng.choice((1e4, 5e5, 1e6)), kind=kind,
                    factor=1.0 if kind == "plain" else rng.uniform(1.5, 64.0), origin=rng.choice((2048, 4096, 8192)))
    heads, dim = rng.choice((1, 2, 3, 4, 5, 8, 8)), rng.choice((64, 128, 128))
    block = rng.choice((1, 1, 16, 16, 32, 64))
    page = 1 if block == 1 and rng.random() < 0.7 else rng.choice([p for p in (16, 32, 64, 128) if p % block == 0])
    if op == "store":
        new_hi = 1 if rng.random() < 0.3 else _log_int(rng, 2, 4096)
        new_lo = 1 if rng.random() < 0.5 else rng.randint(1, new_hi)
        hi = 0 if rng.random() < 0.3 else _log_int(rng, 1, 4096)
        group = rng.choice((0, 1, 2, 3, 4, 7, 8, 16))
        most = min(512, 90_000_000 // (new_hi * heads * dim * (1 + group)), 300_000_000 // ((hi + new_hi) * heads * dim))
        rotary = 0 if group == 0 else rng.choice([r for r in (16, 32, 48, 64, 96, 128, 128) if r <= dim])
        return dict(op=op, heads=heads, group=group, dim=dim, batch=_log_int(rng, 1, max(1, most)),
                    lo=rng.randint(0, hi), hi=hi, new_lo=new_lo, new_hi=new_hi, rotary=rotary,
                    pairs=rng.choice(("half", "interleaved")), block=block, page=page)
    hi = _log_int(rng, 1, 30000)
    lo = rng.randint(1, hi)
    size = 300_000_000 if op == "load" else 700_000_000
    batch = _log_int(rng, 1, max(1, min(256, size // (hi * heads * dim))))
    case = dict(op=op, heads=heads, dim=dim, batch=batch, lo=lo, hi=hi, log=rng.random() < 0.5,
                empty=rng.randint(0, batch // 4), block=block, page=page)
    if op == "decode":
        case["group"] = rng.choice((1, 2, 3, 4, 5, 7, 8, 16))
    return case


def _spread(lo, hi, count, log=False):
    """`count` lengths spread evenly over [lo, hi] (over the logarithm if `log`), the same for every seed."""
    at = [(i + 0.5) / count for i in range(count)]
    if log:
        return [int(round(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * a))) for a in at]
    return [int(round(lo + (hi - lo) * a)) for a in at]


def _lengths(case):
    """Cached tokens of each request (of a store: before it, and the new ones)."""
    if case["op"] == "store":
        new = _spread(case["new_lo"], case["new_hi"], case["batch"])
        return _spread(case["lo"], case["hi"], case["batch"]), [new[(7 * i + 3) % len(new)] for i in range(len(new))]
    live = case["batch"] - case["empty"]
    return _spread(case["lo"], case["hi"], live, case["log"]) + [0] * case["empty"]


def _pow2(e):
    """2.0**e in float32 for whole e from -126 to 127, from its bits: exp2 on the GPU can be a unit off."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _whole(tokens, block):
    return -(-tokens // block)


def work(case):
    if case["op"] == "table":
        return {"bytes": 4 * case["count"] * (1 + case["rotary"]), "flops": 0}
    heads, dim, block = case["heads"], case["dim"], case["block"]
    row = 2 * heads * dim  # one token's K and V in the pool, and in bf16 twice as much
    if case["op"] == "store":  # rotate, quantise and store the new rows; read the blocks that they are in back
        cached, new = _lengths(case)
        tokens = sum(new)
        back = sum(c % block + n for c, n in zip(cached, new))
        blocks = sum(_whole(c + n, block) - c // block for c, n in zip(cached, new))
        q = 4 * heads * case["group"] * dim
        return {"bytes": tokens * (q + 3 * row + 4 + (4 * case["rotary"] + 4 if case["rotary"] else 0))
                + 2 * 2 * heads * blocks + back * (3 * row + 4),
                "flops": 3 * tokens * heads * (1 + case["group"]) * case["rotary"]}
    lens = _lengths(case)
    tokens, blocks = sum(lens), sum(_whole(n, block) for n in lens)
    if case["op"] == "load":
        return {"bytes": tokens * (3 * row + 4) + 2 * heads * blocks, "flops": 0}
    many = heads * case["group"]
    return {"bytes": tokens * (row + 4) + 2 * heads * blocks + case["batch"] * (many * dim * 4 + 4),
            "flops": 4 * tokens * many * dim}


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #
def _values(shape, g):
    """Queries, keys or values as projections give them: normal, some channels wider than others, in bf16."""
    x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, 1.0, generator=g)
    wide = torch.empty(shape[-2:], dtype=torch.float32, device="cuda").normal_(0.0, 0.5, generator=g).exp_()
    return x.mul_(wide).to(torch.bfloat16)


def _table(lens, page, width, g):
    """A page table [B, width] of rows in pages of `page` at random places, and the pool's rows."""
    lens = torch.tensor(lens, device="cuda")
    pages = (lens + page - 1) // page
    first = pages.cumsum(0) - pages
    count = int(pages.sum()) + 64
    order = torch.randperm(count, generator=g, device="cuda")
    j = torch.arange(width, device="cuda")[None, :]
    at = order[(first[:, None] + j // page).clamp_(max=count - 1)] * page + j % page
    return torch.where(j < lens[:, None], at, 0).to(torch.int32), count * page


def _packed(lens):
    ends = torch.tensor(lens, device="cuda").cumsum(0)
    return torch.cat([ends.new_zeros(1), ends]).to(torch.int32)


def _prepare_table(case, g, seed):
    s = {"op": "table", "frequencies": _frequencies(case)}
    if case["spread"]:
        s["positions"] = torch.randint(0, case["spread"], (case["count"],), generator=g, device="cuda",
                                       dtype=torch.int32)
    else:  # a run of positions
        s["positions"] = torch.arange(case["count"], dtype=torch.int32, device="cuda") + seed % 1000
    if own:
        import paged_kv_cache_row_gb300 as mk
        s["rope"] = mk.Rope(case["rotary"], case["base"], kind=case["kind"], factor=case["factor"],
                            original_positions=case["origin"])
    return s


def _prepare_store(case, g):
    heads, dim, block, rotary = case["heads"], case["dim"], case["block"], case["rotary"]
    cached, new = _lengths(case)
    ends = [c + n for c, n in zip(cached, new)]
    width = max(32, -(-max(ends) // 32) * 32)
    table, rows = _table(ends, case["page"], width, g)
    j = torch.arange(width, device="cuda")[None, :]
    as_t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    start, end = as_t(cached)[:, None], as_t(ends)[:, None]
    fresh = (j >= start) & (j < end)
    tokens, q_heads = sum(new), heads * case["group"]
    # q, k and v are slices of one projection's output
    qkv = _values((tokens, q_heads + 2 * heads, dim), g)
    s = {"op": "store", "block": block, "out_loc": table[fresh].contiguous(), "q": qkv[:, :q_heads],
         "k": qkv[:, q_heads:q_heads + heads], "v": qkv[:, q_heads + heads:], "rotary": rotary,
         "interleaved": case["pairs"] == "interleaved"}
    if rotary:
        s["positions"] = j.expand(len(ends), width)[fresh].to(torch.int32)
        turn = dict(rotary=rotary, base=10000.0, kind="plain", factor=1.0, origin=4096)
        angle = torch.arange(max(ends), dtype=torch.float64, device="cuda")[:, None] * torch.tensor(
            _frequencies(turn)[0], dtype=torch.float64, device="cuda")
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["q_out"] = torch.empty((tokens, q_heads, dim), dtype=torch.bfloat16, device="cuda")
    # what is read back: the blocks that the new rows are in, up to the last new row
    back = [n + c % block for c, n in zip(cached, new)]
    at = (start - start % block + j).clamp(max=width - 1)
    s["table"], s["lens"], s["offsets"], s["tokens"] = table.gather(1, at.long()), as_t(back), _packed(back), sum(back)
    return s, rows


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "table":
        return _prepare_table(case, g, seed)
    heads, dim, block = case["heads"], case["dim"], case["block"]
    if case["op"] == "store":
        s, rows = _prepare_store(case, g)
    else:
        lens = _lengths(case)
        turn = torch.randperm(len(lens), generator=g, device="cuda").tolist()
        lens = [lens[i] for i in turn]
        table, rows = _table(lens, case["page"], max(32, -(-max(lens) // 32) * 32), g)
        s = {"op": case["op"], "block": block, "table": table, "tokens": sum(lens), "offsets": _packed(lens),
             "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    rows = -(-rows // 64) * 64
    s["data"] = torch.empty((2, 1, rows, heads, dim), dtype=torch.float8_e4m3fn, device="cuda")
    # the exponents of a block's heads start at a multiple of 4 bytes
    s["scales"] = torch.zeros((2, 1, rows // block, -(-heads // 4) * 4), dtype=torch.uint8, device="cuda")[..., :heads]
    for i in range(2):
        x = _values((rows, heads, dim), g).float().view(rows // block, block, heads, dim)
        e = _needed(x.abs().amax((1, 3)))
        s["data"][i, 0] = (x * _pow2(-e)[:, None, :, None]).to(torch.float8_e4m3fn).view(rows, heads, dim)
        s["scales"][i, 0] = (e + 127).to(torch.uint8)
        del x
    if case["op"] == "decode":
        s["group"] = case["group"]
        s["q"] = (_values((len(s["lens"]), heads * case["group"], dim), g) * 1.5).to(torch.bfloat16)
    if own:
        import paged_kv_cache_row_gb300 as mk
        s["pool"] = mk.KVPoolFP8(s["data"], s["scales"], page_size=case["page"], block_tokens=block)
        if case["op"] == "decode":
            s["workspace"] = mk.decode_workspace_fp8(len(s["lens"]), heads * case["group"], s["pool"])
    return s


# --------------------------------------------------------------------------- #
# plain forms
# --------------------------------------------------------------------------- #
def _frequencies(case):
    """(theta_j, the factor of cos and sin) of the scaling `kind`."""
    n, base, f, origin = case["rotary"], case["base"], case["factor"], case["origin"]
    if case["kind"] == "ntk":  # a larger base: the slowest frequency is f times slower, the fastest the same
        base = base * f ** (n / (n - 2))
    theta = [base ** (-2.0 * j / n) for j in range(n // 2)]
    if case["kind"] == "linear":
        return [t / f for t in theta], 1.0
    if case["kind"] == "bands":  # by how often a frequency turns in the original context: 4 and more as it is, 1 slowed
        keep = [min(1.0, max(0.0, (origin * t / (2 * math.pi) - 1.0) / (4.0 - 1.0))) for t in theta]
        return [(1 - k) * t / f + k * t for k, t in zip(keep, theta)], 1.0
    if case["kind"] == "yarn":  # a ramp over j between the frequencies that turn 32 times and once
        at = [n * math.log(origin / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        lo, hi = max(0, math.floor(at[0])), min(n - 1, math.ceil(at[1]))
        hi = hi if hi > lo else lo + 0.001
        ramp = [min(1.0, max(0.0, (j - lo) / (hi - lo))) for j in range(n // 2)]
        return [r * t / f + (1 - r) * t for r, t in zip(ramp, theta)], 0.1 * math.log(f) + 1.0
    return theta, 1.0


def _needed(top):
    """The smallest e with top <= 448 * 2**e, int32."""
    m, x = torch.frexp(top)  # top = m * 2**x, 0.5 <= m < 1; 448 = 0.875 * 2**9
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(top == 0, LOWEST, e).clamp(LOWEST, HIGHEST)


def _plain_table(s):
    theta, m = s["frequencies"]
    angle = s["positions"].double()[:, None] * torch.tensor(theta, dtype=torch.float64, device="cuda")
    return torch.cat([torch.cos(angle) * m, torch.sin(angle) * m], 1).float()


def _rotate(x, cos, sin, interleaved):
    """x [N, H, d] in float32, the first 2 * cos.shape[1] channels rotated."""
    h = cos.shape[1]
    cos, sin = cos[:, None, :], sin[:, None, :]
    a, b = (x[..., 0:2 * h:2], x[..., 1:2 * h:2]) if interleaved else (x[..., :h], x[..., h:2 * h])
    y, z = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((y, z), -1).flatten(-2) if interleaved else torch.cat((y, z), -1)
    return torch.cat((turned, x[..., 2 * h:]), -1)


def _plain_put(s, i, x):
    """x [N, H, d] in float32 into the rows out_loc of K (i = 0) or V (i = 1)."""
    block, rows = s["block"], s["out_loc"].long()
    data, scales = s["data"][i, 0].view(torch.uint8), s["scales"][i, 0]
    mine, at = torch.unique(rows // block, return_inverse=True)
    inside = torch.arange(block, device="cuda")
    old = data[mine[:, None] * block + inside].view(torch.float8_e4m3fn).float()  # [M, block, H, d]
    top = torch.zeros((len(mine), x.shape[1]), device="cuda")
    top = top.scatter_reduce(0, at[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
    first = torch.full((len(mine),), block, device="cuda").scatter_reduce(0, at, rows % block, "amin")
    so_far = scales[mine].int() - 127
    e = _needed(top)
    e = torch.where((first > 0)[:, None], torch.maximum(e, so_far), e)
    older = (inside[None, :] < first[:, None])[:, :, None, None]
    again = old * _pow2((so_far - e).clamp(min=-126))[:, None, :, None]
    new = torch.where(older, again, old)
    new[at, rows % block] = x * _pow2(-e)[at][:, :, None]
    data[mine[:, None] * block + inside] = new.to(torch.float8_e4m3fn).view(torch.uint8)
    scales[mine] = (e + 127).to(torch.uint8)


def _dequantise(s, i, rows):
    """float32 [..., H, d] of the pool's rows."""
    e = s["scales"][i, 0][rows // s["block"]].int() - 127
    return s["data"][i, 0].view(torch.uint8)[rows].view(torch.float8_e4m3fn).float() * _pow2(e)[..., None]


def _plain_load(s):
    live = torch.arange(s["tokens"], device="cuda")
    r = torch.searchsorted(s["offsets"][1:].long(), live, right=True)
    rows = s["table"][r, live - s["offsets"].long()[r]].long()
    return {"k": _dequantise(s, 0, rows).to(torch.bfloat16), "v": _dequantise(s, 1, rows).to(torch.bfloat16)}


def _plain_store(s):
    k, out = s["k"].float(), {}
    if s["rotary"]:
        cos, sin = s["cos_sin"][s["positions"].long()].chunk(2, 1)
        k = _rotate(k, cos, sin, s["interleaved"])
        out["q"] = _rotate(s["q"].float(), cos, sin, s["interleaved"]).to(torch.bfloat16)
    _plain_put(s, 0, k)
    _plain_put(s, 1, s["v"].float())
    return {**out, **_plain_load(s)}


def _plain_decode(s):
    q, lens = s["q"].float(), s["lens"]
    batch, _, dim = q.shape
    rows = s["table"].long()
    k = _dequantise(s, 0, rows)  # [B, W, H, D]
    q = q.view(batch, -1, s["group"], dim)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) / math.sqrt(dim)  # [B, H, G, W]
    del k
    dead = torch.arange(rows.shape[1], device="cuda")[None, :] >= lens[:, None]
    x = x.masked_fill(dead[:, None, None, :], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-3e38))
    total = p.sum(-1, keepdim=True)
    v = _dequantise(s, 1, rows)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / total.clamp(min=1e-30)
    return o.reshape(batch, -1, dim).to(torch.bfloat16)


def run(state):
    s = state
    if own:
        import paged_kv_cache_row_gb300 as mk
        if s["op"] == "table":
            return mk.minisgl_rope_table(s["rope"], s["positions"])
        if s["op"] == "decode":
            return mk.minisgl_decode_attn_fp8(s["pool"], 0, s["q"], s["table"], s["lens"],
                                              1.0 / math.sqrt(s["q"].shape[2]), workspace=s["workspace"])
        out = {}
        if s["op"] == "store" and s["rotary"]:
            out["q"] = mk.minisgl_rope_store_kv_fp8(s["pool"], 0, s["q"], s["k"], s["v"], s["positions"], s["cos_sin"],
                                                    s["out_loc"], interleaved=s["interleaved"], q_out=s["q_out"])
        elif s["op"] == "store":
            mk.minisgl_store_kv_fp8(s["pool"], 0, s["k"], s["v"], s["out_loc"])
        k, v = mk.minisgl_load_kv_fp8(s["pool"], 0, s["table"], s["lens"], s["offsets"], s["tokens"])
        return {**out, "k": k, "v": v}
    return {"table": _plain_table, "decode": _plain_decode, "store": _plain_store, "load": _plain_load}[s["op"]](s)


# --------------------------------------------------------------------------- #
# the definition in 64 bits
# --------------------------------------------------------------------------- #
def _power(e):
    """2.0**e in float64 for whole e, exactly."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _e4m3(byte):
    """The value of e4m3 bit patterns, from the format: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    b = byte.to(torch.int64)
    e, f = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * _power(e - 7))
    return torch.where(b >= 128, -mag, mag)


def _to_e4m3(x):
    """The e4m3 value nearest to x, the even pattern on a tie."""
    grid = _e4m3(torch.arange(127, device=x.device))
    mid = (grid[1:] + grid[:-1]) / 2
    a = x.abs().contiguous()
    up = torch.searchsorted(mid, a, right=False)  # ties stay below
    up += ((mid[up.clamp(max=len(mid) - 1)] == a) & (up % 2 == 1)).long()
    return torch.copysign(grid[up], x)


def _exact_rows(s, i, rows):
    e = s["scales"][i, 0][torch.div(rows, s["block"], rounding_mode="floor")].long() - 127
    return _e4m3(s["data"][i, 0].view(torch.uint8)[rows]) * _power(e)[..., None]


def _exact_frequencies(case):
    j = np.arange(case["rotary"] // 2, dtype=np.float64)
    f, kind = case["factor"], case["kind"]
    lnb = math.log(case["base"])
    if kind == "ntk":
        lnb += math.log(f) * case["rotary"] / (case["rotary"] - 2)
    theta, m = np.exp(-2.0 * j / case["rotary"] * lnb), 1.0
    if kind == "linear":
        theta = theta / f
    elif kind == "bands":
        wave = 2 * math.pi / theta
        mix = (case["origin"] / wave - 1.0) / 3.0
        theta = np.where(wave < case["origin"] / 4, theta,
                         np.where(wave > case["origin"], theta / f, (1 - mix) * theta / f + mix * theta))
    elif kind == "yarn":
        where = [case["rotary"] / 2 * (math.log(case["origin"] / (2 * math.pi)) - math.log(t)) / lnb for t in (32, 1)]
        lo, hi = max(math.floor(where[0]), 0), min(math.ceil(where[1]), case["rotary"] - 1)
        ramp = np.clip((j - lo) / (hi - lo if hi > lo else 0.001), 0.0, 1.0)
        theta, m = theta * (1 - ramp) + theta / f * ramp, 1 + 0.1 * math.log(f)
    return theta, m


def _exact_table(case, s):
    theta, m = _exact_frequencies(case)
    z = m * np.exp(1j * (s["positions"].cpu().numpy().astype(np.float64)[:, None] * theta))
    return torch.from_numpy(np.concatenate([z.real, z.imag], 1))


def _exact_turned(s, x):
    """x [N, H, d] rotated as complex numbers."""
    x, h = x.double(), s["rotary"] // 2
    row = s["cos_sin"].double()[s["positions"].long()][:, None, :]
    turn = torch.complex(row[..., :h].contiguous(), row[..., h:].contiguous())
    out = x.clone()
    a, b = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if s["interleaved"] else (slice(0, h), slice(h, 2 * h))
    z = torch.complex(x[..., a].contiguous(), x[..., b].contiguous()) * turn
    out[..., a], out[..., b] = z.real, z.imag
    return out


def _exact_put(s, i, x):
    """The values that the rows read back stand for after the store of x."""
    block, rows = s["block"], s["out_loc"].long()
    count, heads = s["scales"].shape[2], x.shape[1]
    home = torch.div(rows, block, rounding_mode="floor")
    top = torch.zeros((count, heads), dtype=torch.float64, device=x.device)
    top.scatter_reduce_(0, home[:, None].expand(-1, heads), x.abs().amax(2), "amax")
    first = torch.full((count,), block, device=x.device).scatter_reduce_(0, home, rows - home * block, "amin")
    need = torch.ceil(torch.log2((top / TOP).clamp(min=2.0 ** LOWEST)))
    need = need.long()
    need += (top > TOP * _power(need)).long() - (top <= TOP * _power(need - 1)).long()
    need = need.clamp(LOWEST, HIGHEST)
    before = s["scales"][i, 0].long() - 127
    e = torch.where((first == 0)[:, None], need, torch.maximum(need, before))
    e = torch.where((first == block)[:, None], before, e)
    live = torch.cat([s["table"][r, :n] for r, n in enumerate(s["lens"].tolist())]).long()
    unit = _power(e)[torch.div(live, block, rounding_mode="floor")][..., None]
    was = _to_e4m3(_exact_rows(s, i, live) / unit) * unit
    where = torch.full((s["data"].shape[2],), -1, device=x.device)
    where[rows] = torch.arange(len(rows), device=x.device)
    new = where[live] >= 0
    was[new] = _to_e4m3(x[where[live][new]] / unit[new]) * unit[new]
    return was


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "table":
        return _exact_table(case, s)
    lens = s["lens"].tolist()
    if s["op"] == "store":
        q, k = (_exact_turned(s, s["q"]), _exact_turned(s, s["k"])) if s["rotary"] else (None, s["k"].double())
        out = {} if q is None else {"q": q}
        return {**out, "k": _exact_put(s, 0, k), "v": _exact_put(s, 1, s["v"].double())}
    if s["op"] == "load":
        rows = torch.cat([s["table"][r, :n].long() for r, n in enumerate(lens)])
        return {"k": _exact_rows(s, 0, rows), "v": _exact_rows(s, 1, rows)}
    heads, dim = s["data"].shape[3], s["q"].shape[2]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for r, n in enumerate(lens):
        if n:
            rows = s["table"][r, :n].long()
            k, v = _exact_rows(s, 0, rows).transpose(0, 1), _exact_rows(s, 1, rows).transpose(0, 1)
            q = s["q"][r].double().view(heads, -1, dim)
            out[r] = (torch.softmax(q @ k.transpose(1, 2) * dim ** -0.5, -1) @ v).view(-1, dim)
    return out
