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
