"""The 8-bit pool's store and load with enough tokens that their kernels reach
their steady states: blocks that go over several tiles, pieces asked for ahead,
units of several heads, windows at their widest.  The launch rules are restated
here, so that a test whose sizes no longer reach such a state fails.

The references are the definitions in torch on the GPU, in 64 bits where a value
is rounded; tests/fp8_ref.py has them in numpy for small sizes."""
import numpy as np
import pytest
import torch

import paged_kv_cache_row_gb300 as mk

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_row_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def pow2(e):
    """2.0**e in float64 for whole e, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def value(code):
    return code.view(torch.float8_e4m3fn).double()


def element(x):
    """e4m3 bytes of x, at most 448 in size: nearest, ties to even."""
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def needed(top):
    """The smallest e with top <= 448 * 2^e, from -120 to 119."""
    m, x = torch.frexp(top)
    return torch.where(top == 0, -120, torch.where(m <= 0.875, x - 9, x - 8)).clamp(-120, 119)


def values_like(shape, g):
    """bf16 values with channels of different widths."""
    x = torch.empty(shape, device=DEV).normal_(0, 1, generator=g)
    return x.mul_(torch.empty(shape[-2:], device=DEV).normal_(0, 0.5, generator=g).exp_()).bfloat16()


def random_pool(rows, H, d, block, g, page=64):
    """A pool of any elements but NaN under scales from 2^-12 to 2^1."""
    data = torch.randint(0, 254, (2, 1, rows, H, d), dtype=torch.uint8, device=DEV, generator=g)
    data += (data >= 127).to(torch.uint8)
    scales = torch.randint(115, 129, (2, 1, rows // block, -(-H // 4) * 4), dtype=torch.uint8, device=DEV, generator=g)
    return mk.KVPoolFP8(data, scales[..., :H], page, block)


# --------------------------------------------------------------------------- #
# load
# --------------------------------------------------------------------------- #
def load_plan(H, d, total):
    """(tokens of a tile, tokens at a time, blocks) of a call, as launch_load_kv_fp8 has them."""
    columns = 2 * H * d // 16
    toks = 256 // columns if columns < 256 else 1
    threads = min(-(-toks * columns // 32) * 32, 512)
    cap = sms() * (1024 // threads)
    tile = min(max(32, 4 * toks), max(toks, -(-total // cap)))
    return tile, toks, min(cap, -(-total // tile))


LOADS = [(8, 128, 16), (33, 128, 1), (1, 64, 64), (5, 64, 32), (3, 128, 16)]


@pytest.mark.parametrize("first", [0, 8], ids=["32-byte", "16-byte"])
@pytest.mark.parametrize("H,d,block", LOADS, ids=["%d-%d-%d" % c for c in LOADS])
def test_load_many_tiles(H, d, block, first):
    """Blocks that take more than two tiles each, with more pieces than are under
    way at once (but where 32 tokens go at a time), and a ragged last tile; gaps
    between the requests, empty requests, and lengths past the next one's start."""
    g = torch.Generator(device=DEV).manual_seed(H)
    rng = np.random.default_rng(H)
    columns = 2 * H * d // 16
    toks = max(1, 256 // columns)
    most = max(32, 4 * toks)
    total = int(2.4 * most * sms() * (1024 // min(-(-toks * columns // 32) * 32, 512))) + 3
    tile, toks, blocks = load_plan(H, d, total)
    assert tile == most and total > 2 * tile * blocks and total % tile and (toks == 32 or tile > 4 * toks)
    B = 40
    cuts = np.sort(rng.integers(0, total - 5, B - 1))
    offsets = np.concatenate([[3], cuts, [total - 2]])
    offsets = np.maximum.accumulate(offsets)
    room = np.diff(offsets)
    lens = np.where(rng.random(B) < 0.3, room, np.maximum(room - rng.integers(0, 50, B), 0))
    lens[5], lens[6] = room[5] + 30, 0
    W = int(lens.max()) + 1
    R = 1 << 14
    pool = random_pool(R, H, d, block, g)
    table = torch.randint(0, R, (B, W), dtype=torch.int32, device=DEV, generator=g)
    # two outputs, 9 wherever nothing is written; the first 16 bytes off a 32-byte border where `first` says so
    n = total * H * d
    out = [torch.full((n + 16,), 9.0, dtype=torch.bfloat16, device=DEV)[at:at + n].view(total, H, d) for at in (first, 0)]
    assert out[0].data_ptr() % 32 == 2 * first and out[1].data_ptr() % 32 == 0
    mk.minisgl_load_kv_fp8(pool, 0, table, i32(lens), i32(offsets), total, out[0], out[1])
    t = np.arange(total)
    r = np.clip(np.searchsorted(offsets, t, "right") - 1, 0, B - 1)
    j = t - offsets[r]
    live = torch.from_numpy((j >= 0) & (j < lens[r]) & (t < offsets[r + 1])).to(DEV)
    rows = table[torch.from_numpy(r).to(DEV), torch.from_numpy(np.clip(j, 0, W - 1)).to(DEV)].long()
    for i in (0, 1):
        e = pool.scales[i, 0][rows // block].int() - 127
        want = (value(pool.data[i, 0][rows]) * pow2(e)[..., None]).bfloat16()
        want[~live] = 9.0
        assert torch.equal(out[i].view(torch.int16), want.view(torch.int16)), "KV"[i]


# --------------------------------------------------------------------------- #
# store
# --------------------------------------------------------------------------- #
def store_plan(H, d, block, n):
    """(log2 of a window's tokens, heads of a unit) of a call, as launch_runs has them."""
    warps = {16: 1, 32: d // 64, 64: d // 32}[block]
    resident, groups = 4 * sms(), 4 // warps

    def units(win, chunks):
        return 2 * -(-n // (1 << win)) * chunks
    win = 0
    while 1 << win < block and units(win + 1, H) >= 2 * resident * groups:
        win += 1
    chunks = H
    while chunks > 1 and units(win, (chunks + 1) // 2) >= 8 * resident * groups:
        chunks = (chunks + 1) // 2
    return win, -(-H // chunks)


def some_tokens(H, d, block, heads):
    """The fewest tokens (to 5 %) whose units have `heads` heads and windows of a whole block."""
    n = 1000
    while store_plan(H, d, block, n) != (block.bit_length() - 1, heads):
        n = int(n * 1.05)
        assert n < 400000
    return n + 17


def requests(n, block, rng):
    """Rows of n tokens of requests that go on behind 0 to 130 cached ones, in pages of 64 anywhere; the pool's rows."""
    rows, at, page = [], 0, 64
    starts = []
    while at < n:
        m = min(int(rng.choice([1, 2, 33, 64, 500, 1500, 4000])), n - at)
        starts.append((int(rng.integers(0, 131)), m))
        at += m
    pages = [-(-(c + m) // page) for c, m in starts]
    order = rng.permutation(sum(pages) + 3)
    first = 0
    for (c, m), k in zip(starts, pages):
        j = np.arange(c, c + m)
        rows.append(order[first + j // page] * page + j % page)
        first += k
    rows = np.concatenate(rows)
    assert len(np.unique(rows)) == len(rows) == n
    return rows, len(order) * page


def first_rows(rows, block):
    """For each token whether a run begins with it."""
    fresh = np.ones(len(rows), bool)
    fresh[1:] = (rows[1:] != rows[:-1] + 1) | (rows[1:] % block == 0)
    return fresh


def old_rows(pool, i, rows):
    """(first run row in its block, or 0) of every block that the rows touch."""
    block = pool.block_tokens
    off = torch.zeros(pool.num_rows // block, dtype=torch.int64, device=DEV)
    at = torch.from_numpy(rows[first_rows(rows, block)]).to(DEV)
    off[at // block] = at % block
    return off


def moved(codes, e_old, e_new, off, block):
    """The rows before a block's run under the block's new scale."""
    R = codes.shape[0]
    r = torch.arange(R, device=DEV)
    grown = (r % block < off[r // block])[:, None] & (e_new > e_old)[r // block]
    down = pow2((e_old - e_new).clamp(max=0))[r // block][..., None]
    return torch.where(grown[..., None], element(value(codes) * down), codes)


# (KV heads, d, block, heads of a unit): the last unit of a token's heads is shorter
STORES = [(5, 64, 64, 2), (5, 64, 16, 3), (5, 128, 16, 2), (7, 128, 16, 4), (5, 128, 32, 2), (5, 64, 32, 3), (3, 128, 64, 2),
          (7, 128, 64, 2)]


@pytest.mark.parametrize("H,d,block,heads", STORES, ids=["%d-%d-%d-%d" % c for c in STORES])
def test_store_units_of_several_heads(H, d, block, heads):
    rng = np.random.default_rng(H * d + block)
    g = torch.Generator(device=DEV).manual_seed(block)
    n = some_tokens(H, d, block, heads)
    assert H % heads
    rows, R = requests(n, block, rng)
    pool = random_pool(R, H, d, block, g)
    x = [values_like((n, H, d), g) for _ in range(2)]
    before = pool.data.clone(), pool.scales.clone()
    mk.minisgl_store_kv_fp8(pool, 0, x[0], x[1], i32(rows))
    for i in (0, 1):
        check_exact(pool, i, rows, x[i], before[0][i, 0], before[1][i, 0])


def check_exact(pool, i, rows, x, codes, scales):
    block, H = pool.block_tokens, pool.num_kv_heads
    at = torch.from_numpy(rows).to(DEV)
    off, e_old = old_rows(pool, i, rows), scales.int() - 127
    top = torch.zeros((pool.num_rows // block, H), device=DEV)
    top.index_reduce_(0, at // block, x.float().abs().amax(2), "amax")
    touched = torch.zeros(len(top), dtype=torch.bool, device=DEV)
    touched[at // block] = True
    need = needed(top)
    e = torch.where((off > 0)[:, None], torch.maximum(need, e_old), need)
    e = torch.where(touched[:, None], e, e_old)
    assert torch.equal(pool.scales[i, 0].int() - 127, e)
    assert ((e > e_old) & (off > 0)[:, None]).any()  # some older rows are moved
    want = moved(codes, e_old, e, off, block)
    want[at] = element(x.double() * pow2(-e)[at // block][..., None])
    # what lies behind a block's run means nothing; the calls leave it
    assert torch.equal(pool.data[i, 0], want)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("H,d,block,heads", STORES, ids=["%d-%d-%d-%d" % c for c in STORES])
def test_rope_store_units_of_several_heads(H, d, block, heads, interleaved):
    """K's state lies between that of the ends of the interval that fp32 allows, and q within half a step of bf16."""
    rng = np.random.default_rng(H * d + block + 1)
    g = torch.Generator(device=DEV).manual_seed(block + 1)
    n, Hq, rotary = some_tokens(H, d, block, heads), 3, d // 2 if interleaved else d
    rows, R = requests(n, block, rng)
    at = torch.from_numpy(rows).to(DEV)
    pool = random_pool(R, H, d, block, g)
    qkv = values_like((n, Hq + 2 * H, d), g)
    q, k, v = qkv.split([Hq, H, H], 1)
    before = pool.data.clone(), pool.scales.clone()
    cache = mk.minisgl_rope_table(mk.Rope(rotary), i32(range(5000)))
    pos = torch.randint(0, 5000, (n,), dtype=torch.int32, device=DEV, generator=g)
    out = mk.minisgl_rope_store_kv_fp8(pool, 0, q, k, v, pos, cache, i32(rows), interleaved=interleaved,
                                       q_out=torch.empty((n, Hq, d), dtype=torch.bfloat16, device=DEV))
    check_exact(pool, 1, rows, v, before[0][1, 0], before[1][1, 0])
    y, off = rotated(q, cache[pos.long()], interleaved)
    assert ((out.double() - y).abs() <= 2.0 ** -8 * y.abs() + 2 * off).all()
    del y, off
    # one rounding of a product and one of the sum: 2^-23 of the terms
    y, slack = rotated(k, cache[pos.long()], interleaved)
    blk, first, e_old = at // block, old_rows(pool, 0, rows), before[1][0, 0].int() - 127
    e = pool.scales[0, 0].int() - 127
    ends = []
    for s in (-1, 1):
        top = torch.zeros((R // block, H), dtype=torch.float64, device=DEV)
        top.index_reduce_(0, blk, (y.abs() + s * slack).clamp(min=0).amax(2), "amax")
        ends.append(torch.where((first > 0)[:, None], torch.maximum(needed(top), e_old), needed(top)))
    assert ((e >= ends[0]) & (e <= ends[1]))[blk].all()
    untouched = torch.ones(R // block, dtype=torch.bool, device=DEV)
    untouched[blk] = False
    assert torch.equal(e[untouched], e_old[untouched])
    unit = pow2(e)[blk][..., None]
    got = value(pool.data[0, 0][at])
    # (through fp32: it keeps the order, and the kernel's values are fp32)
    low, high = (value(element(((y + s * slack) / unit).clamp(-448, 448))) for s in (-1, 1))
    assert ((got >= low) & (got <= high)).all()
    want = moved(before[0][0, 0], e_old, e, first, block)
    assert ((e > e_old) & (first > 0)[:, None]).any()
    want[at] = pool.data[0, 0][at]
    assert torch.equal(pool.data[0, 0], want)


def rotated(x, cos_sin, interleaved):
    """x turned in 64 bits, and 2^-23 of the terms' magnitudes together."""
    x = x.double()
    h = cos_sin.shape[1] // 2
    c, s = cos_sin[:, None, :h].double(), cos_sin[:, None, h:].double()
    a, b = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    y, off = x.clone(), torch.zeros_like(x)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    off[..., a] = 2.0 ** -23 * ((x[..., a] * c).abs() + (x[..., b] * s).abs())
    off[..., b] = 2.0 ** -23 * ((x[..., b] * c).abs() + (x[..., a] * s).abs())
    return y, off
