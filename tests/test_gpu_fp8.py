"""GPU tests of the 8-bit pool's calls and the rotary tables against the plain
64-bit definitions in tests/fp8_ref.py.  Stored bytes and loaded values must be
equal (behind a rotation: the bytes of a value within fp32's roundings); decode
attention stays within bounds counted from its roundings (fp4_ref.decode_bound)."""
import math
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_kv_cache_row_gb300 as mk
from tests import fp4_ref
from tests import fp8_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_row_gb300 import build
    build.build()
    assert torch.cuda.is_available()


@pytest.fixture(autouse=True)
def _no_wait_ran_out():
    yield
    assert mk.minisgl_debug_timeout_count() == 0


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def kv_like(shape, seed, scale=1.0):
    """bf16 values with channels of different widths."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=shape) * np.exp(0.5 * rng.normal(size=shape[-2:])) * scale
    return torch.from_numpy(x).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def pool_state(pool, layer=0):
    """(codes [R, H, d], exponents [blocks, H]) of K and of V, as numpy."""
    d, s = pool.data.cpu().numpy(), pool.scales.cpu().numpy().astype(int) - 127
    return [(d[i, layer].copy(), s[i, layer].copy()) for i in (0, 1)]


def pool_values(pool, layer=0):
    return [ref.values(c, e, pool.block_tokens) for c, e in pool_state(pool, layer)]


def new_pool(rows, H, d, block, layers=1, page=None):
    """A pool full of bytes that nobody wrote (no NaN, so that differences show)."""
    pool = mk.KVPoolFP8.zeros(layers, rows, H, d, page or max(block, 1), block)
    pool.data.fill_(0x55)
    pool.scales.fill_(100)
    return pool


# --------------------------------------------------------------------------- #
# rotary tables
# --------------------------------------------------------------------------- #
# cos and sin: the argument (at most pi/4) is off by 3 roundings, 3 * 2^-25, the
# polynomial by 2^-28 and its last step's rounding 2^-25, the product with the
# factor 2^-25: together below 2^-22 of it.
TABLE_TOL = 2.0 ** -22


@pytest.mark.parametrize("rotary", [16, 48, 64, 128, 256])
@pytest.mark.parametrize("kind", ["plain", "linear", "ntk", "bands", "yarn"])
def test_rope_table(rotary, kind):
    rope = mk.Rope(rotary, 10000.0, kind, factor=1.0 if kind == "plain" else 8.0, original_positions=4096)
    rng = np.random.default_rng(rotary)
    pos = np.concatenate([np.arange(40), rng.integers(0, 1 << 20, 70), rng.integers(-(1 << 31), 1 << 31, 50),
                          [-1, -(1 << 31), (1 << 31) - 1]])
    got = f64(mk.minisgl_rope_table(rope, i32(pos)))
    want = ref.table(rope.turns, rope.attention_factor, pos)
    assert np.abs(got - want).max() <= TABLE_TOL * rope.attention_factor
    assert np.array_equal(got[0, :rotary // 2], np.full(rotary // 2, np.float64(np.float32(rope.attention_factor))))
    assert (got[0, rotary // 2:] == 0).all()


@pytest.mark.parametrize("n", [1, 2, 7, 31, 33, 1000, 40000])
def test_rope_table_lengths(n):
    rope = mk.Rope(96)
    pos = (np.arange(n) * 37) % 10007
    buf = torch.full((n + 2, 96), 7.0, device=DEV)
    out = buf[1:n + 1]
    assert mk.minisgl_rope_table(rope, i32(pos), out=out) is out
    angle = pos[:, None] * np.array(ref.frequencies(96, 10000.0)[0])
    assert np.abs(f64(out) - np.concatenate([np.cos(angle), np.sin(angle)], 1)).max() <= TABLE_TOL + 1e-9
    assert (buf[0] == 7).all() and (buf[n + 1] == 7).all()


def test_rope_table_is_the_workloads_table():
    """Beside the table that the bf16 store is tested with (angles in fp32: off by 2^-24 of them, 2 roundings)."""
    import workloads
    want = workloads.rope_cos_sin_cache(128, 2000).double().numpy()
    got = f64(mk.minisgl_rope_table(mk.Rope(128), i32(range(2000))))
    assert np.abs(got - want).max() <= 2000 * 2.0 ** -22 + TABLE_TOL


def test_rope_table_of_nothing():
    assert mk.minisgl_rope_table(mk.Rope(64), i32([])).shape == (0, 64)


def test_rope_table_small_angles_keep_their_bits():
    """sin of a small angle is the angle: within 2^-21 of it, however slow the frequency."""
    rope = mk.Rope(128, 1e6, "linear", factor=64.0)
    got = f64(mk.minisgl_rope_table(rope, i32([1, 3])))[:, 64:]
    want = np.sin(np.array([[1.0], [3.0]]) * np.array(rope.turns) / 2.0 ** 64 * 2 * math.pi)
    assert (np.abs(got - want) <= 2.0 ** -21 * np.abs(want)).all()


# --------------------------------------------------------------------------- #
# store
# --------------------------------------------------------------------------- #
def check_state(pool, want, layer=0):
    for (c, e), (wc, we), name in zip(pool_state(pool, layer), want, "KV"):
        assert np.array_equal(e, we), (name, np.argwhere(e != we)[:5])
        assert np.array_equal(c, wc), (name, np.argwhere(c != wc)[:5])


def store_and_check(pool, rows, k, v, layer=0, k_dev=None, v_dev=None):
    """The call against the definition, on the pool's whole state.  Bytes of a
    block behind its run mean nothing: they are taken over."""
    want = pool_state(pool, layer)
    for (c, e), x in zip(want, (k, v)):
        ref.store(c, e, list(rows), f64(x), pool.block_tokens)
    mk.minisgl_store_kv_fp8(pool, layer, k.to(DEV) if k_dev is None else k_dev, v.to(DEV) if v_dev is None else v_dev,
                            i32(rows))
    check_state(pool, want, layer)


def some_runs(rng, blocks, block, count):
    """Rows of `count` runs in different blocks: from anywhere to anywhere in them."""
    rows = []
    for b in rng.permutation(blocks)[:count]:
        first = int(rng.integers(0, block))
        rows += list(range(b * block + first, b * block + int(rng.integers(first + 1, block + 1))))
    return rows


@pytest.mark.parametrize("H,d", [(1, 64), (2, 64), (3, 128), (5, 64), (8, 128)])
@pytest.mark.parametrize("block", [1, 16, 32, 64])
def test_store_bytes(H, d, block):
    rng = np.random.default_rng(H * d + block)
    pool = new_pool(40 * block + 3, H, d, block)
    for step in range(4):
        rows = some_runs(rng, 40, block, 25)
        k, v = (kv_like((len(rows), H, d), 10 * step + i, 4.0 ** (step - 1)) for i in (1, 2))
        store_and_check(pool, rows, k, v)


@pytest.mark.parametrize("block", [16, 32, 64])
def test_store_token_by_token(block):
    """Decode steps: one row of each block per call, larger and smaller values in turn, to the blocks' ends."""
    H, d = 2, 128
    pool = new_pool(6 * block, H, d, block)
    rng = np.random.default_rng(block)
    for t in range(block):
        scale = 2.0 ** rng.integers(-12, 6)
        k, v = (kv_like((6, H, d), 100 * t + i, scale) for i in (1, 2))
        store_and_check(pool, [b * block + t for b in range(6)], k, v)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 100, 3001])
@pytest.mark.parametrize("block", [1, 16, 32, 64])
def test_store_one_long_request(n, block):
    """Consecutive rows from every kind of first row, over many windows and blocks."""
    H, d = 2, 64
    first = {1: 0, 16: 5, 32: 31, 64: 1}[block]
    pool = new_pool(first + n + 1, H, d, block)
    store_and_check(pool, range(first, first + n), kv_like((n, H, d), n), kv_like((n, H, d), n + 1))


def test_store_many_tokens():
    """Windows at their widest, pages in random order."""
    H, d, block, page = 8, 128, 16, 64
    lens = [700, 1, 64, 65, 1300, 2047, 15, 16, 17]
    pages = np.random.default_rng(0).permutation(sum(-(-n // page) for n in lens))
    rows, at = [], 0
    for n in lens:
        own = pages[at:at + -(-n // page)]
        at += len(own)
        rows += [int(own[j // page]) * page + j % page for j in range(n)]
    pool = new_pool(len(pages) * page, H, d, block, page=page)
    store_and_check(pool, rows, kv_like((len(rows), H, d), 1), kv_like((len(rows), H, d), 2))


def test_store_blocks_in_any_order():
    """Runs of one block are one run only if they follow one another: rows that
    go on in the next block of the pool, or end and start there, are others."""
    block = 16
    rows = list(range(40, 48)) + list(range(48, 52)) + [16] + list(range(0, 3)) + [65, 66] + [17 + 64]
    pool = new_pool(96, 3, 128, block)
    store_and_check(pool, rows, kv_like((len(rows), 3, 128), 5), kv_like((len(rows), 3, 128), 6))


def test_store_strided_rows_and_page_first_pool():
    """K and V cut out of a projection's output; pool axes in another order; another layer."""
    L, R, H, d, block = 3, 64, 5, 64, 16
    data = torch.full((R, 2, L, H, d), 0x55, dtype=torch.uint8, device=DEV).permute(1, 2, 0, 3, 4)
    scales = torch.full((R // block, 2, L, 8), 100, dtype=torch.uint8, device=DEV)[..., :H].permute(1, 2, 0, 3)
    pool = mk.KVPoolFP8(data, scales, 16, block)
    qkv = kv_like((30, 4 * H, d), 3).to(DEV)
    k, v = qkv[:, 2 * H:3 * H], qkv[:, 3 * H:]
    others = [pool_state(pool, i) for i in (0, 2)]
    store_and_check(pool, list(range(7, 27)) + list(range(48, 58)), k.cpu(), v.cpu(), 1, k, v)
    for i, want in zip((0, 2), others):
        check_state(pool, want, i)


@pytest.mark.parametrize("block", [1, 16])
def test_store_every_largest_value(block):
    """Every positive bf16, finite or not, as a block's largest; its scale and the element itself."""
    x = torch.arange(0, 0x7F80, 1 if block == 1 else 7, dtype=torch.int16).view(torch.bfloat16)
    n = len(x)
    k = torch.zeros((n, 1, 64), dtype=torch.bfloat16)
    k[:, 0, 17] = x
    k[:, 0, 40] = -x / 3
    v = -k.flip(-1)
    pool = new_pool(n * block, 1, 64, block)
    store_and_check(pool, [i * block for i in range(n)], k, v)


def test_store_ties_and_subnormals():
    """Every border between two elements, under the block's largest value 448, and its neighbours in bf16."""
    mid = (ref.E4M3[1:] + ref.E4M3[:-1]) / 2
    x = torch.from_numpy(np.concatenate([mid, -mid, ref.E4M3])).to(torch.bfloat16)
    near = torch.cat([x, (x.view(torch.int16) + 1).view(torch.bfloat16), (x.view(torch.int16) - 1).view(torch.bfloat16)])
    near = near[near.float().abs() <= 448]
    k = torch.zeros((-(-len(near) // 127), 1, 128), dtype=torch.bfloat16)
    for i in range(len(k)):
        part = near[i * 127:(i + 1) * 127]
        k[i, 0, :len(part)] = part
        k[i, 0, 127] = 448
    for block in (1, 16):
        for power in (0, -100, 100):
            y = (k.double() * 2.0 ** power).to(torch.bfloat16)
            store_and_check(new_pool(len(k) * block, 1, 128, block), [i * block for i in range(len(k))], y, -y)


@pytest.mark.parametrize("block", [1, 16, 64])
def test_store_nan_and_infinity(block):
    """NaN and infinities become NaN where they are; the others keep the scale they need."""
    n = 24
    k, v = kv_like((n, 3, 128), 1), kv_like((n, 3, 128), 2)
    k[3, 1, 5], k[7, 2, 100], v[9, 0, 64], v[0, 1, 0] = math.nan, math.inf, -math.inf, math.nan
    v[20] = math.inf
    k[11] = math.nan
    pool = new_pool(64, 3, 128, block)
    store_and_check(pool, range(8, 8 + n), k, v)
    assert np.isnan(pool_values(pool)[0][8 + 11]).all() and np.isnan(pool_values(pool)[1][8 + 20]).all()


def test_store_zeros():
    pool = new_pool(32, 2, 64, 16)
    z = torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    store_and_check(pool, range(16, 21), z, -z)
    store_and_check(pool, range(21, 24), kv_like((3, 2, 64), 1), z[:3])
    assert (pool_state(pool)[1][1][1] == -120).all()


def test_store_older_rows_under_far_larger_values():
    """From the smallest scale to the largest in one step: the older rows vanish, a NaN among them stays."""
    pool = new_pool(16, 1, 128, 16)
    a, b = kv_like((4, 1, 128), 1, 1e-30), kv_like((1, 1, 128), 2, 1e30)
    a[2, 0, 3] = math.nan
    store_and_check(pool, range(4), a, a)
    store_and_check(pool, [4], b, b)
    got = pool_values(pool)[0][:4]
    assert np.isnan(got[2, 0, 3]) and np.nansum(np.abs(got)) == 0


@pytest.mark.parametrize("block", [1, 16])
def test_store_padding_rows_leave_the_others_alone(block):
    """Many tokens on the dummy row, between and behind the others; rows outside the pool are clamped to its ends."""
    H, d = 8, 128
    pool = new_pool(12 * block, H, d, block)
    dummy = 11 * block + block // 2
    rows = [2 * block] + [dummy] * 40 + [5 * block] + [dummy] * 300
    k, v = kv_like((len(rows), H, d), 1), kv_like((len(rows), H, d), 2)
    want = pool_state(pool)
    for (c, e), x in zip(want, (k, v)):
        ref.store(c, e, [2 * block], f64(x)[:1], block)
        ref.store(c, e, [5 * block], f64(x)[41:42], block)
    mk.minisgl_store_kv_fp8(pool, 0, k.to(DEV), v.to(DEV), i32(rows))
    for (c, e), (wc, we) in zip(pool_state(pool), want):
        assert np.array_equal(c[:11 * block], wc[:11 * block]) and np.array_equal(e[:11], we[:11])
    before = pool_state(pool)
    mk.minisgl_store_kv_fp8(pool, 0, k[:3].to(DEV), v[:3].to(DEV), i32([-5, 12 * block, 1 << 30]))
    for (c, e), (wc, we) in zip(pool_state(pool), before):
        assert np.array_equal(c[block:11 * block], wc[block:11 * block]) and np.array_equal(e[1:11], we[1:11])


def test_store_nothing():
    pool = new_pool(32, 2, 64, 16)
    want = pool_state(pool)
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    mk.minisgl_store_kv_fp8(pool, 0, e, e, i32([]))
    mk.minisgl_rope_store_kv_fp8(pool, 0, e, e, e, i32([]), torch.zeros(4, 64, device=DEV), i32([]))
    check_state(pool, want)


@pytest.mark.parametrize("H,d,block", [(33, 128, 16), (130, 64, 1), (70, 64, 64)])
def test_store_and_load_many_heads(H, d, block):
    n = 70
    pool = new_pool(n + 10, H, d, block, page=64)
    rows = list(range(3, 3 + n))
    store_and_check(pool, rows, kv_like((n, H, d), 1), kv_like((n, H, d), 2))
    k, v = mk.minisgl_load_kv_fp8(pool, 0, i32([rows]), i32([n]), i32([0, n]), n)
    for got, want in zip((k, v), pool_values(pool)):
        assert np.array_equal(f64(got), want[rows])


# --------------------------------------------------------------------------- #
# store with a rotation
# --------------------------------------------------------------------------- #
def check_rotated_store(pool, before, rows, x, off):
    """K's state against the definition for values within `off` of x: e and the
    bytes lie between those of the interval's ends."""
    block = pool.block_tokens
    (codes, exps), _ = pool_state(pool)
    for i, row, n in ref.runs(rows, block):
        b, skip = row // block, row % block
        a, t = np.abs(x[i:i + n]), off[i:i + n]
        lo, hi = (ref.needed(np.maximum(y, 0).max((0, 2))) for y in (a - t, a + t))
        if skip:
            lo, hi = np.maximum(lo, before[1][b]), np.maximum(hi, before[1][b])
        e = exps[b]
        assert (e >= lo).all() and (e <= hi).all(), (row, e, lo, hi)
        unit = 2.0 ** e.astype(float)[:, None]
        got = ref.value(codes[row:row + n]) * unit
        low, high = (ref.value(ref.element(y / unit)) * unit for y in (x[i:i + n] - t, x[i:i + n] + t))
        assert (got >= low).all() and (got <= high).all(), row
        if skip:  # the rows before the run, under the scale that the block has now
            was = ref.value(before[0][row - skip:row]) * 2.0 ** (before[1][b] - e)[:, None]
            assert np.array_equal(ref.value(codes[row - skip:row]), ref.value(ref.element(was)))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary,d", [(16, 64), (48, 64), (64, 64), (32, 128), (64, 128), (112, 128), (128, 128)])
@pytest.mark.parametrize("block", [1, 16, 64])
@pytest.mark.parametrize("in_place", [False, True])
def test_rope_store(interleaved, rotary, d, block, in_place):
    rng = np.random.default_rng(rotary + d + block)
    H, Hq = 2, 6
    pool = new_pool(20 * block, H, d, block)
    # older rows everywhere, then runs that begin inside blocks
    start = np.arange(20 * block)
    mk.minisgl_store_kv_fp8(pool, 0, kv_like((len(start), H, d), 1, 0.3).to(DEV),
                            kv_like((len(start), H, d), 2, 0.3).to(DEV), i32(start))
    rows = some_runs(rng, 20, block, 13)
    n = len(rows)
    qkv = kv_like((n, Hq + 2 * H, d), 7).to(DEV)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
    keep = [f64(t) for t in (q, k, v)]
    pos = rng.integers(0, 5000, n)
    cache = mk.minisgl_rope_table(mk.Rope(rotary), i32(range(5000)))
    before, (vc, ve) = pool_state(pool)
    q_out = None if in_place else torch.full((n, Hq, d), 9.0, dtype=torch.bfloat16, device=DEV)
    out = mk.minisgl_rope_store_kv_fp8(pool, 0, q, k, v, i32(pos), cache, i32(rows), interleaved=interleaved,
                                       q_out=q_out)
    assert out is (q if in_place else q_out)
    turn = f64(cache)[pos]
    want, off = ref.rotate(keep[0], turn, interleaved)
    # half a step of bf16 (2^-8 of the value), the fp32 rotation, and bf16's smallest half step
    assert (np.abs(f64(out) - want) <= 2.0 ** -8 * np.abs(want) + 2 * off + 2.0 ** -134).all()
    assert np.array_equal(f64(k), keep[1]) and np.array_equal(f64(v), keep[2])
    if not in_place:
        assert np.array_equal(f64(q), keep[0])
    if rotary < d:
        assert np.array_equal(f64(out)[..., rotary:], keep[0][..., rotary:])
    check_rotated_store(pool, before, rows, *ref.rotate(keep[1], turn, interleaved))
    ref.store(vc, ve, rows, keep[2], block)
    got = pool_state(pool)[1]
    assert np.array_equal(got[0], vc) and np.array_equal(got[1], ve)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary,d", [(16, 64), (48, 64), (64, 64), (32, 128), (112, 128), (128, 128)])
@pytest.mark.parametrize("in_place", [False, True])
def test_rope_store_blocks_of_32(interleaved, rotary, d, in_place):
    test_rope_store(interleaved, rotary, d, 32, in_place)


def test_rope_store_is_the_bf16_calls_rotation():
    """Half-split pairs over the whole head: q as minisgl_rope_store_kv gives it, bit for bit."""
    H, Hq, d, n = 2, 8, 128, 50
    q, k, v = (kv_like((n, h, d), 20 + i).to(DEV) for i, h in enumerate((Hq, H, H)))
    cache = mk.minisgl_rope_table(mk.Rope(d), i32(range(1000)))
    pos, rows = i32(np.arange(n) * 13), i32(range(n))
    wide = mk.KVPool(torch.zeros((2, 1, n, H, d), dtype=torch.bfloat16, device=DEV))
    want = mk.minisgl_rope_store_kv(wide, 0, q.clone(), k, v, pos, cache, rows)
    pool = new_pool(n, H, d, 1)
    got = mk.minisgl_rope_store_kv_fp8(pool, 0, q, k, v, pos, cache, rows, q_out=torch.empty_like(q))
    assert torch.equal(got, want)


def test_rope_store_infinities_and_positions_outside():
    """A rotation of an infinity is NaN in both channels; positions are clamped to the table."""
    pool = new_pool(16, 1, 64, 16)
    k = kv_like((3, 1, 64), 1)
    k[1, 0, 5] = math.inf
    cache = mk.minisgl_rope_table(mk.Rope(64), i32(range(1, 11)))
    q = kv_like((3, 1, 64), 2).to(DEV)
    out = mk.minisgl_rope_store_kv_fp8(pool, 0, q, k.to(DEV), k.to(DEV), i32([-7, 3, 99]), cache, i32([0, 1, 2]),
                                       q_out=torch.empty_like(q))
    got = pool_values(pool)[0]
    assert np.isnan(got[1, 0, [5, 37]]).all() and np.isnan(got[:3]).sum() == 2
    want, off = ref.rotate(f64(q), f64(cache)[[0, 3, 9]], False)
    assert (np.abs(f64(out) - want) <= 2.0 ** -8 * np.abs(want) + 2 * off).all()


def test_rope_store_with_a_steps_own_table():
    """A row of the table for each token: the same as the whole table by position."""
    H, d, n = 2, 64, 40
    rope = mk.Rope(64, kind="yarn", factor=16.0, original_positions=4096)
    pos = i32(np.random.default_rng(0).integers(0, 60000, n))
    q, k, v = (kv_like((n, h, d), h).to(DEV) for h in (4, 2, 2))
    pools = [new_pool(n, H, d, 16) for _ in range(2)]
    a = mk.minisgl_rope_store_kv_fp8(pools[0], 0, q, k, v, pos, mk.minisgl_rope_table(rope, i32(range(60000))),
                                     i32(range(n)), q_out=torch.empty_like(q))
    b = mk.minisgl_rope_store_kv_fp8(pools[1], 0, q, k, v, i32(range(n)), mk.minisgl_rope_table(rope, pos),
                                     i32(range(n)), q_out=torch.empty_like(q))
    assert torch.equal(a, b)
    check_state(pools[0], pool_state(pools[1]))


@pytest.mark.parametrize("block", [1, 16])
@pytest.mark.parametrize("first", ["q", "q_out"])
def test_rope_store_into_another_slice_of_the_same_buffer(first, block):
    """q, q_out, k and v are columns of one buffer, q before q_out and behind it."""
    H, Hq, d, n = 2, 6, 64, 37
    buf = kv_like((n, 2 * Hq + 2 * H, d), 4).to(DEV)
    left, right, k, v = buf.split([Hq, Hq, H, H], 1)
    q, q_out = (left, right) if first == "q" else (right, left)
    kept = buf.clone()
    pool, twin = new_pool(64, H, d, block), new_pool(64, H, d, block)
    cache, rows = mk.minisgl_rope_table(mk.Rope(32), i32(range(100))), i32(range(7, 7 + n))
    want = mk.minisgl_rope_store_kv_fp8(twin, 0, q.clone(), k.clone(), v.clone(), rows, cache, rows)
    assert mk.minisgl_rope_store_kv_fp8(pool, 0, q, k, v, rows, cache, rows, q_out=q_out) is q_out
    at = slice(Hq, 2 * Hq) if first == "q" else slice(0, Hq)
    kept[:, at] = want
    assert torch.equal(buf, kept)
    check_state(pool, pool_state(twin))


def test_rope_store_one_token_in_place_whatever_its_strides():
    """The strides of one token mean nothing."""
    pool, twin = new_pool(16, 2, 64, 16), new_pool(16, 2, 64, 16)
    q, k, v = (kv_like((1, h, 64), h).to(DEV) for h in (4, 2, 3))
    v = v[:, :2]
    cache, at = mk.minisgl_rope_table(mk.Rope(64), i32(range(9))), i32([5])
    want = mk.minisgl_rope_store_kv_fp8(twin, 0, q.clone(), k, v, at, cache, at)
    lib = mk.load_library()
    assert lib.minisgl_rope_store_kv_fp8(pool._ref, 0, q.data_ptr(), 4, 256, q.data_ptr(), 4096, k.data_ptr(),
                                         v.data_ptr(), 128, 192, at.data_ptr(), cache.data_ptr(), 9, 64, 0, at.data_ptr(),
                                         1, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(q, want)
    check_state(pool, pool_state(twin))


# --------------------------------------------------------------------------- #
# load
# --------------------------------------------------------------------------- #
def filled_pool(rows, H, d, block, seed, layers=1, scale=1.0):
    pool = new_pool(rows, H, d, block, layers)
    for layer in range(layers):
        k, v = (kv_like((rows, H, d), seed + 2 * layer + i, scale).to(DEV) for i in (0, 1))
        mk.minisgl_store_kv_fp8(pool, layer, k, v, i32(range(rows)))
    return pool


@pytest.mark.parametrize("H,d", [(1, 64), (3, 64), (8, 128), (5, 128)])
@pytest.mark.parametrize("block", [1, 32])
def test_load_rows(H, d, block):
    """Raw rows in any order, gaps between the requests, a short total, lengths past the table and below zero."""
    rng = np.random.default_rng(H)
    R, W, stride = 320, 50, 64
    pool = filled_pool(R, H, d, block, 3, layers=2)
    lens = [50, 0, 17, 99, -3, 1, 33]
    offsets = [2, 52, 60, 77, 120, 121, 125, 150]
    total = 140
    buf = i32(rng.integers(0, R, (len(lens), stride)))
    table = buf[:, :W]
    pad = torch.full((2, total, 2 * H, d), 9.0, dtype=torch.bfloat16, device=DEV)
    k, v = pad[0, :, :H], pad[1, :, H:]
    mk.minisgl_load_kv_fp8(pool, 1, table, i32(lens), i32(offsets), total, k, v)
    want = np.full((2, total, 2 * H, d), 9.0)
    pt = table.cpu().numpy()
    for r, n in enumerate(lens):
        for j in range(min(max(n, 0), W)):
            at = offsets[r] + j
            if at < min(total, offsets[r + 1]):
                want[0, at, :H] = pool_values_cached(pool, 1)[0][pt[r, j]]
                want[1, at, H:] = pool_values_cached(pool, 1)[1][pt[r, j]]
    assert np.array_equal(f64(pad), want)


_cache = {}


def pool_values_cached(pool, layer):
    key = (id(pool), layer)
    if key not in _cache:
        _cache.clear()
        _cache[key] = (pool, pool_values(pool, layer))
    return _cache[key][1]


def test_load_every_value():
    """Every element under every scale that a store gives, and NaN."""
    pool = new_pool(240, 2, 128, 1)
    codes = torch.arange(256, dtype=torch.uint8, device=DEV).view(2, 128)
    pool.data[:] = codes
    pool.scales[:] = torch.arange(7, 247, dtype=torch.uint8, device=DEV)[:, None]
    k, v = mk.minisgl_load_kv_fp8(pool, 0, i32([range(240)]), i32([240]), i32([0, 240]), 240)
    for got, want in zip((k, v), pool_values(pool)):
        assert np.array_equal(f64(got), want, equal_nan=True)


def test_load_many_short_requests():
    rng = np.random.default_rng(1)
    B, H, d = 700, 2, 64
    pool = filled_pool(512, H, d, 16, 5)
    lens = rng.integers(0, 9, B)
    off = np.concatenate([[0], np.cumsum(lens)])
    table = rng.integers(0, 512, (B, 8))
    k, v = mk.minisgl_load_kv_fp8(pool, 0, i32(table), i32(lens), i32(off), int(off[-1]))
    rows = np.concatenate([table[r, :n] for r, n in enumerate(lens)])
    for got, want in zip((k, v), pool_values(pool)):
        assert np.array_equal(f64(got), want[rows])


# --------------------------------------------------------------------------- #
# decode
# --------------------------------------------------------------------------- #
def check_decode(pool, q, table, lens, sm, layer=0, out=None, vmax=None, **kw):
    """Against 64 bits.  What is lost below 2^-32 of the largest contribution is
    at most 2^-32 of a block's 448 * 2^e, below twice the block's largest value
    where its scale is the one it needs (else vmax is given)."""
    k, v = pool_values(pool, layer)
    pt = table.cpu().numpy()
    n = np.clip(np.asarray(lens), 0, pt.shape[1])
    got = mk.minisgl_decode_attn_fp8(pool, layer, q, table, i32(lens), sm, out=out, **kw)
    want, mag, top = fp4_ref.decode(f64(q), k, v, pt, n, sm)
    bound = fp4_ref.decode_bound(want, mag, top, 2 * np.abs(v).max() if vmax is None else vmax, max(1, int(n.max())))
    err = np.abs(f64(got) - want)
    assert (err <= bound).all(), (float(err.max()), float((err - bound).max()))
    return got


def case(B, Hq, H, d, block, lens, seed, width=None, scale=1.0):
    rng = np.random.default_rng(seed)
    width = width or max(32, -(-max(lens) // 32) * 32)
    R = max(64, min(4096, B * width))
    pool = filled_pool(R, H, d, block, seed, scale=scale)
    table = i32(rng.integers(0, R, (B, width)))
    return pool, kv_like((B, Hq, d), seed + 9, 1.5).to(DEV), table


SHAPES = [(1, 1, 64), (4, 1, 128), (8, 2, 64), (16, 1, 128), (16, 8, 128), (32, 8, 128), (15, 5, 64), (7, 7, 128),
          (12, 3, 128), (9, 1, 64), (96, 6, 64), (64, 4, 128), (10, 10, 64), (22, 11, 128), (51, 17, 128), (25, 25, 64),
          (144, 9, 128)]


@pytest.mark.parametrize("Hq,H,d", SHAPES, ids=["%d-%d-%d" % s for s in SHAPES])
@pytest.mark.parametrize("block", [1, 16])
def test_decode_head_layouts(Hq, H, d, block):
    lens = [1, 31, 0, 32, 33, 700, 64, 5, 129]
    pool, q, table = case(len(lens), Hq, H, d, block, lens, Hq + H)
    check_decode(pool, q, table, lens, d ** -0.5)


@pytest.mark.parametrize("G", [2, 9])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H", list(range(1, 19)) + [21, 32])
def test_decode_every_count_of_heads(H, d, G):
    """Blocks of heads of every size, and last blocks with one head less up to one head."""
    lens = [1, 97, 0, 260]
    pool, q, table = case(len(lens), G * H, H, d, 16, lens, H)
    check_decode(pool, q, table, lens, d ** -0.5)


@pytest.mark.parametrize("Hq,H,d", [(8, 2, 64), (16, 8, 128), (32, 2, 128), (11, 11, 128), (7, 7, 64)])
def test_decode_short_tables(Hq, H, d):
    """Tables of one tile: streams are left whole, empty ones too."""
    lens = [0, 1, 31, 32, 7, 0]
    pool, q, table = case(6, Hq, H, d, 16, lens, 3, width=32)
    out = torch.full_like(q, 7.0)
    check_decode(pool, q, table, lens, d ** -0.5, out=out)
    assert (out[[0, 5]] == 0).all()


@pytest.mark.parametrize("B", [75, 76, 77, 151, 152, 153, 304, 305])
@pytest.mark.parametrize("width", [160, 256, 288])
def test_decode_batches_near_the_number_of_groups(B, width):
    rng = np.random.default_rng(B + width)
    lens = rng.integers(0, width + 1, B)
    lens[B // 2] = width
    pool, q, table = case(B, 8, 4, 64, 64, lens, B, width=width)
    check_decode(pool, q, table, lens, 0.125)


@pytest.mark.parametrize("split", [1, 32, 48, 100, 10 ** 6])
@pytest.mark.parametrize("max_splits", [2, 5, 64, 256])
def test_decode_split_counts(split, max_splits):
    lens = [1000, 33, 0, 65, 2]
    pool, q, table = case(5, 8, 2, 128, 16, lens, 5)
    check_decode(pool, q, table, lens, 0.09, split_tokens=split, max_splits=max_splits)


@pytest.mark.parametrize("Hq,H,d,block,lens", [(16, 2, 128, 64, [20000, 3]), (8, 8, 64, 1, [9001]), (32, 1, 128, 16, [12345]),
                                               (4, 4, 128, 16, [1] * 40 + [5000])],
                         ids=["two", "one", "one-head", "among-short"])
def test_decode_long(Hq, H, d, block, lens):
    if Hq // H > 16:
        Hq = 16
    pool, q, table = case(len(lens), Hq, H, d, block, lens, 11)
    check_decode(pool, q, table, lens, d ** -0.5)


def test_decode_many_requests():
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 60, 4096)
    pool, q, table = case(4096, 2, 1, 64, 16, lens, 6, width=64)
    check_decode(pool, q, table, lens, 0.125)


def test_decode_lengths_past_the_table_and_below_zero():
    pool, q, table = case(4, 4, 2, 64, 16, [64], 8, width=64)
    check_decode(pool, q, table, [1000, -3, 65, 2 ** 31 - 1], 0.125)


def test_decode_sharp_scores():
    """Scores far apart, the largest last, first and in between: the references move in steps and all at once."""
    B, H, d, n = 3, 2, 128, 200
    pool = new_pool(B * n, H, d, 1)
    k, v = kv_like((B * n, H, d), 1), kv_like((B * n, H, d), 2)
    ramp = np.concatenate([np.linspace(0, 3, n), np.linspace(3, 0, n), np.random.default_rng(0).uniform(0, 3, n)])
    k = (f64(k) * ramp[:, None, None])
    q = kv_like((B, 4, d), 3, 4.0)
    k = torch.from_numpy(k + 0.0).to(torch.bfloat16)
    mk.minisgl_store_kv_fp8(pool, 0, k.to(DEV), v.to(DEV), i32(range(B * n)))
    table = i32(np.arange(B * n).reshape(B, n))
    for sm in (0.09, -0.09, 1.0):
        check_decode(pool, q.to(DEV), table, [n, n, n], sm)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("power", [16, 23, 27, 31, 60, 112])
def test_decode_scores_of_any_size(power, sign):
    """One token's score is 2^power, the others' zero (or minus it): the sum is one token's value, or n - 1 tokens'."""
    d, n = 64, 70
    k = torch.zeros((n, 1, d), dtype=torch.bfloat16)
    k[33, 0, 0] = 2.0 ** (power // 2)
    q = torch.zeros((1, 1, d), dtype=torch.bfloat16, device=DEV)
    q[0, 0, 0] = sign * 2.0 ** (power - power // 2)
    v = kv_like((n, 1, d), 5)
    for block in (1, 16):
        pool = new_pool(n, 1, d, block)
        mk.minisgl_store_kv_fp8(pool, 0, k.to(DEV), v.to(DEV), i32(range(n)))
        out = f64(mk.minisgl_decode_attn_fp8(pool, 0, q, i32([range(n)]), i32([n]), 1.0))
        vv = pool_values(pool)[1]
        want = vv[33] if sign > 0 else np.delete(vv, 33, 0).mean(0)
        # weights are equal: exact but for the sum's and output's roundings, 2^-8 and 70 * 2^-24 of the magnitudes
        assert (np.abs(out[0] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -11 * np.abs(vv).max()).all()


@pytest.mark.parametrize("power", [-110, -40, 40, 100])
def test_decode_value_and_key_ranges(power):
    """V by 2^power and K by 2^power with q by 2^-power: the result is the same but for its scale."""
    lens, d = [100, 7, 33], 128
    rng = np.random.default_rng(0)
    k, v, q = kv_like((256, 2, d), 1), kv_like((256, 2, d), 2), kv_like((3, 4, d), 3)
    table = i32(rng.integers(0, 256, (3, 128)))
    outs = []
    for pk, pv in ((0, 0), (power, 0), (0, power)):
        pool = new_pool(256, 2, d, 16)
        kk, vv, qq = ((x.double() * 2.0 ** p).to(torch.bfloat16).to(DEV) for x, p in ((k, pk), (v, pv), (q, -pk)))
        mk.minisgl_store_kv_fp8(pool, 0, kk, vv, i32(range(256)))
        outs.append(f64(mk.minisgl_decode_attn_fp8(pool, 0, qq, table, i32(lens), d ** -0.5)) * 2.0 ** -pv)
    assert np.array_equal(outs[0], outs[1]) and np.array_equal(outs[0], outs[2])


def test_decode_scales_far_apart():
    """Blocks of V that are zero, tiny and huge beside ordinary ones: none of them takes another out of the sum."""
    d, n, block = 64, 96, 16
    k, v = kv_like((n, 1, d), 1), kv_like((n, 1, d), 2)
    v[:16] = 0
    v[16:32] *= 2.0 ** -60
    k[32:48] = 0
    q = kv_like((1, 2, d), 3).to(DEV)
    table, vmax = i32([range(n)]), 0.0
    for huge in (1.0, 2.0 ** 40, 2.0 ** -100):
        v2 = v.clone()
        v2[80:] = (v[80:].double() * huge).to(torch.bfloat16)
        pool = new_pool(n, 1, d, block)
        mk.minisgl_store_kv_fp8(pool, 0, k.to(DEV), v2.to(DEV), i32(range(n)))
        for lens in ([n], [80], [32], [16], [17]):
            got = check_decode(pool, q, table, lens, 0.125)
            if lens == [16]:
                assert (got == 0).all()
    # a weight of one on tiny values, next to weights of nearly nothing on ordinary ones
    k[:] = -8
    k[20] = 8
    q[:] = 8
    pool = new_pool(n, 1, d, block)
    mk.minisgl_store_kv_fp8(pool, 0, k.to(DEV), v.to(DEV), i32(range(n)))
    got = f64(mk.minisgl_decode_attn_fp8(pool, 0, q, table, i32([n]), 1.0))[0, 0]
    want = pool_values(pool)[1][20, 0]  # weights of the others: e^-8192
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want)).all() and np.abs(want).max() > 0


def check_decode_closely(pool, q, table, lens, sm):
    """check_decode with what is lost counted per output: a weight times its
    block's 2^e is in fp16 with the largest of the request and head at 2^7 or
    more, so it is off by 2^-11 of itself or by fp16's last half step, 2^-25:
    2^-32 of the largest, times the element."""
    (kc, ke), (vc, ve) = pool_state(pool)
    k, v = ref.values(kc, ke, pool.block_tokens), ref.values(vc, ve, pool.block_tokens)
    pt, G = table.cpu().numpy(), q.shape[1] // pool.num_kv_heads
    n = np.asarray(lens)
    got = f64(mk.minisgl_decode_attn_fp8(pool, 0, q, table, i32(lens), sm))
    qq = f64(q)
    want, mag, top = fp4_ref.decode(qq, k, v, pt, n, sm)
    bound = fp4_ref.decode_bound(want, mag, top, 0.0, 0)
    for r in range(len(n)):
        rows = pt[r, :n[r]]
        for h in range(q.shape[1]):
            s = sm * k[rows, h // G] @ qq[r, h]
            w = np.exp(s - s.max())
            w *= 2.0 ** ve[rows // pool.block_tokens, h // G] / w.sum()
            bound[r, h] += (1 + 2.0 ** -7) * 2.0 ** -32 * w.max() * np.abs(ref.value(vc[rows, h // G])).sum(0)
    err = np.abs(got - want)
    assert (err <= bound).all(), (float(err.max()), float((err - bound).max()))


@pytest.mark.parametrize("block", [1, 16])
@pytest.mark.parametrize("power", [4, 12, 17, 20, 22, 26, 31, 40])
def test_decode_an_outlier_in_one_channel(power, block):
    """One channel of V is 2^power times the others in one block: the block's
    tokens lose their other channels to the scale (at 2^-18 of the outlier), and
    the other tokens keep theirs as far as fp16 weights under the larger scale do."""
    d, n = 64, 96
    k, v = kv_like((n, 2, d), 1), kv_like((n, 2, d), 2)
    v[40, 0, 7] = 2.0 ** power
    q = kv_like((3, 4, d), 3).to(DEV)
    pool = new_pool(n, 2, d, block)
    mk.minisgl_store_kv_fp8(pool, 0, k.to(DEV), v.to(DEV), i32(range(n)))
    check_decode_closely(pool, q, i32([range(n)] * 3), [n, 32, 41], 0.125)


@pytest.mark.parametrize("Hq,H,d,block", [(8, 2, 64, 16), (16, 8, 128, 1), (16, 1, 128, 64), (15, 5, 128, 32), (9, 3, 64, 1)])
def test_decode_closely(Hq, H, d, block):
    lens = [1, 31, 96, 33, 700, 64, 5, 129]
    pool, q, table = case(len(lens), Hq, H, d, block, lens, Hq + H)
    check_decode_closely(pool, q, table, lens, d ** -0.5)


@pytest.mark.parametrize("huge", [1.0, 2.0 ** 40, 2.0 ** -100])
def test_decode_scales_far_apart_closely(huge):
    """Contexts without the block that is far larger are held to their own values."""
    d, n, block = 64, 96, 16
    k, v = kv_like((n, 1, d), 1), kv_like((n, 1, d), 2)
    v[:16] = 0
    v[16:32] *= 2.0 ** -60
    k[32:48] = 0
    v[80:] = (v[80:].double() * huge).to(torch.bfloat16)
    pool = new_pool(n, 1, d, block)
    mk.minisgl_store_kv_fp8(pool, 0, k.to(DEV), v.to(DEV), i32(range(n)))
    q = kv_like((5, 2, d), 3).to(DEV)
    check_decode_closely(pool, q, i32([range(n)] * 5), [n, 80, 32, 16, 17], 0.125)


def test_decode_nan_stays_in_its_head():
    lens = [40, 100]
    pool, q, table = case(2, 8, 4, 64, 1, lens, 3)
    rows = table[0, :40].tolist()
    only = [r for r in rows if r not in set(table[1, :100].tolist())][0]
    pool.data[1, 0, only, 2, 5] = 0x7F
    out = mk.minisgl_decode_attn_fp8(pool, 0, q, table, i32(lens), 0.125)
    nan = torch.isnan(out).nonzero().tolist()
    assert sorted(nan) == [[0, 4, 5], [0, 5, 5]]


def test_decode_rows_behind_the_length_are_not_read():
    """NaN rows and rows outside the pool behind a request's end change nothing."""
    lens = [33, 1, 70]
    pool, q, table = case(3, 8, 4, 128, 16, lens, 5, width=96)
    want = mk.minisgl_decode_attn_fp8(pool, 0, q, table, i32(lens), 0.1)
    bad = (set(range(pool.num_rows)) - set(r for i, n in enumerate(lens) for r in table[i, :n].tolist())).pop()
    pool.data[:, :, bad] = 0x7F
    for junk in (bad, -5, 1 << 30):
        t = table.clone()
        for i, n in enumerate(lens):
            t[i, n:] = junk
        assert torch.equal(mk.minisgl_decode_attn_fp8(pool, 0, q, t, i32(lens), 0.1), want)


def test_decode_table_stride_workspace_and_out():
    lens = [300, 45]
    pool, q, table = case(2, 8, 4, 64, 16, lens, 3)
    wide = torch.full((2, 777), -1, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    ws = mk.decode_workspace_fp8(2, 8, pool, 7)
    ws.fill_(0xFF)
    out = torch.empty_like(q)
    a = check_decode(pool, q, wide[:, :table.shape[1]], lens, 0.125, out=out, workspace=ws)
    assert a is out
    assert torch.equal(a, mk.minisgl_decode_attn_fp8(pool, 0, q, table, i32(lens), 0.125, workspace=ws))


def test_decode_is_the_same_every_time():
    rng = np.random.default_rng(4)
    lens = rng.integers(1, 3000, 40)
    pool, q, table = case(40, 32, 8, 128, 16, lens, 6)
    ws = mk.decode_workspace_fp8(40, 32, pool)
    first = mk.minisgl_decode_attn_fp8(pool, 0, q, table, i32(lens), 0.09, workspace=ws)
    for _ in range(5):
        assert torch.equal(first, mk.minisgl_decode_attn_fp8(pool, 0, q, table, i32(lens), 0.09, workspace=ws))


@pytest.mark.parametrize("slots", [2, 5], ids=["packed", "spread"])
@pytest.mark.parametrize("H,d", [(5, 128), (3, 64), (9, 64)])
def test_scales_beside_each_other_and_apart(H, d, slots):
    """K's and V's scales of a block next to one another, or with other bytes between them."""
    block, R, room = 16, 256, -(-H // 4) * 4
    buf = torch.full((R // block, slots, room), 0xFF, dtype=torch.uint8, device=DEV)
    scales = buf[:, :2, :H].permute(1, 0, 2)[:, None]
    pool = mk.KVPoolFP8(torch.zeros((2, 1, R, H, d), dtype=torch.uint8, device=DEV), scales, 16, block)
    k, v = kv_like((R, H, d), 1).to(DEV), kv_like((R, H, d), 2).to(DEV)
    mk.minisgl_store_kv_fp8(pool, 0, k, v, i32(range(R)))
    assert (buf[:, 2:] == 0xFF).all() and (buf[:, :2, H:] == 0xFF).all()
    table = i32(np.random.default_rng(0).integers(0, R, (3, 96)))
    check_decode(pool, kv_like((3, 2 * H, d), 5).to(DEV), table, [96, 3, 50], 0.1)


def test_rows_past_32_bit_offsets():
    """A pool whose last rows lie past 2^32 bytes, in all calls."""
    H, d, block = 8, 128, 16
    R = (1 << 22) + 1024  # rows of 1 KB
    data = torch.empty((1, 1, 1), dtype=torch.uint8, device=DEV)
    data = torch.empty((2, 1, R, H, d), dtype=torch.uint8, device=DEV)
    scales = torch.full((2, 1, R // block, H), 100, dtype=torch.uint8, device=DEV)
    pool = mk.KVPoolFP8(data, scales, 16, block)
    n, first = 100, R - 128 + 3
    rows = list(range(first, first + n))
    q, k, v = (kv_like((n, h, d), h).to(DEV) for h in (16, 8, 8))
    cache = mk.minisgl_rope_table(mk.Rope(128), i32(range(n)))
    mk.minisgl_rope_store_kv_fp8(pool, 0, q, k, v, i32(range(n)), cache, i32(rows))
    small = mk.KVPoolFP8(data[:, :, R - 128:].clone(), scales[:, :, -8:].clone(), 16, block)
    kk, vv = mk.minisgl_load_kv_fp8(pool, 0, i32([rows]), i32([n]), i32([0, n]), n)
    values = pool_values(small)
    assert np.array_equal(f64(kk), values[0][3:3 + n]) and np.array_equal(f64(vv), values[1][3:3 + n])
    a = mk.minisgl_decode_attn_fp8(pool, 0, q[:1], i32([rows]), i32([n]), 0.1)
    near = i32([range(3, 3 + n)])
    assert torch.equal(a, check_decode(small, q[:1].contiguous(), near, [n], 0.1))


def off_by_16_bytes(shape, seed=None):
    """A bf16 tensor of this shape whose first element is 16 bytes past a 256-byte border."""
    n = int(np.prod(shape))
    t = torch.full((n + 8,), 9.0, dtype=torch.bfloat16, device=DEV)[8:].view(shape)
    if seed is not None:
        t.copy_(kv_like(shape, seed))
    assert t.data_ptr() % 32 == 16
    return t


@pytest.mark.parametrize("block", [1, 16, 64])
@pytest.mark.parametrize("H,d", [(3, 64), (2, 128)])
def test_everything_aligned_to_16_bytes_only(H, d, block):
    """Rows of the pool 16 bytes longer than they need be, scales 4 bytes past a
    border, and every tensor 16 bytes past one."""
    R, n, Hq = 192, 100, 2 * H
    raw = torch.full((2 * R * (H * d + 16) + 16,), 0x55, dtype=torch.uint8, device=DEV)[16:]
    data = raw.as_strided((2, 1, R, H, d), (R * (H * d + 16), 0, H * d + 16, d, 1))
    nb = R // block
    sraw = torch.full((2 * nb * 12 + 16,), 100, dtype=torch.uint8, device=DEV)[4:]
    scales = sraw.as_strided((2, 1, nb, H), (nb * 12, 0, 12, 1))
    pool = mk.KVPoolFP8(data, scales, 64, block)
    q, k, v = (off_by_16_bytes((n, h, d), h + i) for i, h in enumerate((Hq, H, H)))
    rows = list(range(40, 40 + n))
    cache = mk.minisgl_rope_table(mk.Rope(d), i32(range(500)))
    pos = np.arange(n) * 3
    (before, (vc, ve)) = pool_state(pool)
    kept = f64(q)
    out = mk.minisgl_rope_store_kv_fp8(pool, 0, q, k, v, i32(pos), cache, i32(rows), interleaved=True,
                                       q_out=off_by_16_bytes((n, Hq, d)))
    want, off = ref.rotate(kept, f64(cache)[pos], True)
    assert (np.abs(f64(out) - want) <= 2.0 ** -8 * np.abs(want) + 2 * off).all()
    check_rotated_store(pool, before, rows, *ref.rotate(f64(k), f64(cache)[pos], True))
    ref.store(vc, ve, rows, f64(v), block)
    got = pool_state(pool)[1]
    assert np.array_equal(got[0], vc) and np.array_equal(got[1], ve)
    assert (raw.as_strided((2, R, 16), (R * (H * d + 16), H * d + 16, 1), raw.storage_offset() + H * d) == 0x55).all()
    store_and_check(pool, rows, k.cpu(), v.cpu(), 0, k, v)
    ko, vo = off_by_16_bytes((n + 1, H, d)), off_by_16_bytes((n + 1, H, d))
    mk.minisgl_load_kv_fp8(pool, 0, i32([rows]), i32([n]), i32([0, n]), n + 1, ko, vo)
    for got, vals in zip((ko, vo), pool_values(pool)):
        assert np.array_equal(f64(got[:n]), vals[rows]) and (got[n] == 9).all()
    table = i32(np.random.default_rng(0).integers(40, 40 + n, (3, 133)))
    qd = off_by_16_bytes((3, Hq, d), 5)
    check_decode(pool, qd, table, [133, 1, 64], 0.1, out=off_by_16_bytes((3, Hq, d)))


@pytest.mark.parametrize("B,Hq,H,d,long", [(160, 8, 4, 128, 20000), (320, 6, 2, 64, 9000), (90, 16, 8, 128, 5000)])
def test_decode_a_long_request_among_many(B, Hq, H, d, long):
    """More partials of one request than a warp has under way in the merge of many rows."""
    lens = np.random.default_rng(B).integers(0, 40, B)
    lens[B // 3] = long
    pool, q, table = case(B, Hq, H, d, 16, lens, B)
    check_decode(pool, q, table, lens, d ** -0.5)
    check_decode(pool, q, table, lens, d ** -0.5, max_splits=200)


@pytest.mark.parametrize("width", [1, 31, 33, 65, 1000])
def test_decode_table_widths(width):
    lens = [width, 1, 0, max(1, width // 2)]
    pool, q, table = case(4, 8, 4, 64, 32, lens, width, width=width)
    check_decode(pool, q, table, lens, 0.125)


def test_calls_without_requests():
    pool = new_pool(32, 2, 64, 16)
    none, q = i32([]), torch.empty((0, 4, 64), dtype=torch.bfloat16, device=DEV)
    assert mk.minisgl_decode_attn_fp8(pool, 0, q, torch.zeros((0, 32), dtype=torch.int32, device=DEV), none, 0.1).shape == (0, 4, 64)
    k, v = mk.minisgl_load_kv_fp8(pool, 0, torch.zeros((0, 32), dtype=torch.int32, device=DEV), none, i32([0]), 0)
    assert k.shape == v.shape == (0, 2, 64)
    k = torch.full((3, 2, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    mk.minisgl_load_kv_fp8(pool, 0, i32([[1, 2]]), i32([0]), i32([0, 0]), 3, k, k.clone())
    assert (k == 5).all()


def test_store_without_queries():
    """num_q_heads 0: K and V alone, rotated."""
    pool, twin = new_pool(32, 2, 64, 16), new_pool(32, 2, 64, 16)
    k, v, q = (kv_like((20, h, 64), h).to(DEV) for h in (2, 3, 4))
    v = v[:, :2].contiguous()
    cache, rows = mk.minisgl_rope_table(mk.Rope(32), i32(range(50))), i32(range(5, 25))
    mk.minisgl_rope_store_kv_fp8(pool, 0, q[:, :0].contiguous(), k, v, rows, cache, rows)
    mk.minisgl_rope_store_kv_fp8(twin, 0, q, k, v, rows, cache, rows)
    check_state(pool, pool_state(twin))


# --------------------------------------------------------------------------- #
# streams, graphs, refusals
# --------------------------------------------------------------------------- #
def test_calls_on_a_named_stream():
    lens = [60, 33]
    pool, q, table = case(2, 8, 4, 64, 16, lens, 3)
    want = mk.minisgl_decode_attn_fp8(pool, 0, q, table, i32(lens), 0.125)
    loaded = mk.minisgl_load_kv_fp8(pool, 0, table, i32(lens), i32([0, 60, 93]), 93)
    rope = mk.Rope(64)
    rows = mk.minisgl_rope_table(rope, i32(range(50)))
    side = torch.cuda.Stream()
    n, off = i32(lens), i32([0, 60, 93])
    pos = i32(range(50))
    torch.cuda.synchronize()
    assert torch.equal(mk.minisgl_rope_table(rope, pos, stream=side), rows)
    got = mk.minisgl_decode_attn_fp8(pool, 0, q, table, n, 0.125, stream=side)
    k, v = mk.minisgl_load_kv_fp8(pool, 0, table, n, off, 93, stream=side)
    twin = new_pool(64, 4, 64, 16)
    mk.minisgl_store_kv_fp8(twin, 0, k[:60], v[:60], pos[:0].new_tensor(range(60)), stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(k, loaded[0]) and torch.equal(v, loaded[1])


@pytest.mark.parametrize("block", [1, 16, 32])
def test_stores_on_a_named_stream(block):
    """Their rows are made on that stream, behind work that takes a while: a call on another stream would store what was there before."""
    H, Hq, d, n = 3, 6, 64, 60
    side = torch.cuda.Stream()
    x = [kv_like((n, h, d), 10 + h).to(DEV) for h in (Hq, H, H)]
    q, k, v = (torch.zeros_like(t) for t in x)
    rows, cache = i32(range(4, 4 + n)), mk.minisgl_rope_table(mk.Rope(d), i32(range(99)))
    pools = [new_pool(64, H, d, block) for _ in range(4)]
    want = mk.minisgl_rope_store_kv_fp8(pools[0], 0, x[0].clone(), x[1], x[2], rows, cache, rows)
    mk.minisgl_store_kv_fp8(pools[1], 0, x[1], x[2], rows)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms
        for a, b in zip((q, k, v), x):
            a.copy_(b)
    got = mk.minisgl_rope_store_kv_fp8(pools[2], 0, q, k, v, rows, cache, rows, stream=side)
    mk.minisgl_store_kv_fp8(pools[3], 0, k, v, rows, stream=side)
    side.synchronize()
    assert got is q and torch.equal(q, want)
    check_state(pools[2], pool_state(pools[0]))
    check_state(pools[3], pool_state(pools[1]))


@pytest.mark.parametrize("block", [1, 16, 32, 64])
def test_captured_stores_and_load(block):
    """Both stores and the load captured, and replayed while rows, values and lengths change in place."""
    H, Hq, d, n, page = 3, 6, 128, 90, 64
    rng = np.random.default_rng(block)
    pools = [new_pool(20 * page, H, d, block, layers=2, page=page) for _ in range(2)]
    cache = mk.minisgl_rope_table(mk.Rope(64), i32(range(20 * page)))
    q, k, v, out = (torch.zeros((n, h, d), dtype=torch.bfloat16, device=DEV) for h in (Hq, H, H, Hq))
    rows, pos, lens, off = i32(range(n)), i32(range(n)), i32([0, 0]), i32([0, 0, 0])
    table, ko, vo = i32(np.zeros((2, n))), torch.zeros_like(k), torch.zeros_like(k)

    def step(pool, q, k, v, out, ko, vo):
        mk.minisgl_rope_store_kv_fp8(pool, 0, q, k, v, pos, cache, rows, interleaved=True, q_out=out)
        mk.minisgl_store_kv_fp8(pool, 1, k, v, rows)
        mk.minisgl_load_kv_fp8(pool, 1, table, lens, off, n, ko, vo)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(pools[0], q, k, v, out, ko, vo)
    for turn in range(4):
        a = int(rng.integers(1, n))  # two runs of rows in pages of their own
        first = rng.permutation(9)[:2] * 2 * page + rng.integers(0, 30, 2)
        r = np.concatenate([first[0] + np.arange(a), first[1] + np.arange(n - a)])
        for t, x in ((rows, i32(r)), (pos, i32(rng.integers(0, 20 * page, n))), (lens, i32([a, n - a])), (off, i32([0, a, n]))):
            t.copy_(x)
        table[0, :a], table[1, :n - a] = rows[:a], rows[a:]
        for t, h in ((q, Hq), (k, H), (v, H)):
            t.copy_(kv_like((n, h, d), 10 * turn + h, 1.5 ** turn))
        g.replay()
        twin = [torch.empty_like(t) for t in (out, ko, vo)]
        step(pools[1], q, k, v, *twin)
        assert all(torch.equal(x, y) for x, y in zip((out, ko, vo), twin))
        for layer in (0, 1):
            check_state(pools[0], pool_state(pools[1], layer), layer)
        assert np.array_equal(f64(ko), pool_values(pools[0], 1)[0][r])


FIRST_USE_CAPTURED = """
import torch, paged_kv_cache_row_gb300 as mk
d = "cuda"
rope = mk.Rope(64)
pool = mk.KVPoolFP8.zeros(1, 64, 2, 64, 16)
q, k, v = (torch.randn(4, h, 64, device=d).bfloat16() for h in (4, 2, 2))
at = torch.tensor([0, 1, 2, 16], dtype=torch.int32, device=d)
pos = torch.tensor([0, 1, 2, 0], dtype=torch.int32, device=d)
table = torch.tensor([[0, 1, 2, 0], [16, 0, 0, 0]], dtype=torch.int32, device=d)
lens = torch.tensor([3, 1], dtype=torch.int32, device=d)
off = torch.tensor([0, 3, 4], dtype=torch.int32, device=d)
ws = mk.decode_workspace_fp8(2, 4, pool)
def step():
    rows = mk.minisgl_rope_table(rope, pos)
    t = mk.minisgl_rope_store_kv_fp8(pool, 0, q, k, v, at * 0 + torch.arange(4, dtype=torch.int32, device=d), rows, at,
                                     q_out=torch.empty_like(q))
    return (rows, t, mk.minisgl_decode_attn_fp8(pool, 0, t[2:].contiguous(), table, lens, 0.1, workspace=ws),
            *mk.minisgl_load_kv_fp8(pool, 0, table, lens, off, 4))
side = torch.cuda.Stream()
with torch.cuda.stream(side):
    torch.arange(4, dtype=torch.int32, device=d) * 0 + at  # torch's own first uses
side.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = step()
g.replay()
torch.cuda.synchronize()
want = step()
assert all(torch.equal(a, b) for a, b in zip(got, want))
assert mk.minisgl_debug_timeout_count() == 0
print("same")
"""


def test_first_use_may_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST_USE_CAPTURED], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_binding_refusals():
    pool = new_pool(64, 4, 64, 16)
    k, q = kv_like((8, 4, 64), 1).to(DEV), kv_like((8, 8, 64), 2).to(DEV)
    rows, cache = i32(range(8)), torch.zeros(32, 64, device=DEV)
    table, lens = i32(np.zeros((8, 32))), i32([1] * 8)

    def bad(f, *a, **kw):
        with pytest.raises(mk.MinisglError):
            f(*a, **kw)
    s, r, g, a, t = (mk.minisgl_store_kv_fp8, mk.minisgl_rope_store_kv_fp8, mk.minisgl_load_kv_fp8,
                     mk.minisgl_decode_attn_fp8, mk.minisgl_rope_table)
    bad(s, pool, 1, k, k, rows), bad(s, pool, -1, k, k, rows), bad(s, pool, 0, k.float(), k, rows)
    bad(s, pool, 0, k[:7], k, rows), bad(s, pool, 0, k, k[:, :3], rows), bad(s, pool, 0, k, k, rows.long())
    bad(s, pool, 0, k, k, rows.cpu()), bad(s, pool, 0, k.cpu(), k, rows), bad(s, pool, 0, k.transpose(1, 2), k, rows)
    bad(s, pool, 0, k, k, i32(range(16))[::2])
    bad(r, pool, 0, q, k, k, rows, cache.half(), rows), bad(r, pool, 0, q, k, k, rows, cache[:, :40], rows)
    bad(r, pool, 0, q, k, k, rows, torch.zeros(32, 128, device=DEV), rows)
    bad(r, pool, 0, q, k, k, rows, torch.zeros(0, 64, device=DEV), rows), bad(r, pool, 0, q, k, k, rows[:7], cache, rows)
    bad(r, pool, 0, q[:7], k, k, rows, cache, rows), bad(r, pool, 0, q.float(), k, k, rows, cache, rows)
    bad(r, pool, 0, q.view(8, 4, 128), k, k, rows, cache, rows)
    bad(r, pool, 0, q, k, k, rows, cache, rows, q_out=torch.empty_like(q[:, :4]))
    bad(r, pool, 0, q, k, k, rows, cache, rows, q_out=q.float()), bad(r, pool, 0, q, k, k, rows, cache.cpu(), rows)
    both = torch.zeros(9, 8, 64, dtype=torch.bfloat16, device=DEV)
    bad(r, pool, 0, both[:8], k, k, rows, cache, rows, q_out=both[1:])
    bad(g, pool, 0, table, lens[:7], i32(range(9)), 8), bad(g, pool, 0, table, lens, i32(range(8)), 8)
    bad(g, pool, 0, table, lens, i32(range(9)), -1), bad(g, pool, 0, table.t(), lens, i32(range(9)), 8)
    bad(g, pool, 0, table, lens, i32(range(9)), 8, k.float()), bad(g, pool, 0, table, lens, i32(range(9)), 8, k[:7], k)
    bad(a, pool, 0, q[:, :6], table, lens, 0.1), bad(a, pool, 0, q, table[:7], lens, 0.1)
    bad(a, pool, 0, q, table, lens[:7], 0.1), bad(a, pool, 0, q, table, lens, 0.1, out=q[:7])
    bad(a, pool, 0, q, table, lens, 0.1, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    bad(a, pool, 0, q, table, lens, 0.1, workspace=torch.empty(1 << 22, dtype=torch.uint8))
    bad(a, pool, 0, q, table, lens, 0.1, split_tokens=-1)
    bad(t, mk.Rope(64), rows.cpu()), bad(t, mk.Rope(64), rows.long()), bad(t, mk.Rope(64), rows, out=cache)
    bad(t, mk.Rope(64), rows, out=cache[:8].half())
    # pools
    data = torch.zeros((2, 1, 64, 5, 64), dtype=torch.uint8, device=DEV)
    ok = torch.zeros((2, 1, 4, 8), dtype=torch.uint8, device=DEV)[..., :5]
    mk.KVPoolFP8(data.view(torch.float8_e4m3fn), ok, 16, 16)
    bad(mk.KVPoolFP8, data[0], ok, 16, 16), bad(mk.KVPoolFP8, data.float(), ok, 16, 16)
    bad(mk.KVPoolFP8, data, ok.float(), 16, 16), bad(mk.KVPoolFP8, data, ok, 16, 8), bad(mk.KVPoolFP8, data, ok, 24, 16)
    bad(mk.KVPoolFP8, data, ok[:, :, :3], 16, 16), bad(mk.KVPoolFP8, data, ok.cpu(), 16, 16)
    bad(mk.KVPoolFP8, data[..., ::2], ok, 16, 16)
    tight = torch.zeros((2, 1, 4, 5), dtype=torch.uint8, device=DEV)
    bad(mk.KVPoolFP8, data, tight, 16, 16)  # no room behind the last block's five scales


# --------------------------------------------------------------------------- #
# the calls together
# --------------------------------------------------------------------------- #
class Engine:
    """One layer of a serving engine over the 8-bit pool, by the public calls:
    slots, rotation and store, and extend or decode attention."""

    def __init__(self, B, W, pages, page, Hq, H, d, seed):
        self.B, self.page, self.Hq, self.H, self.d = B, page, Hq, H, d
        self.dummy = pages * page
        self.pool = mk.KVPoolFP8.zeros(1, (pages + 1) * page, H, d, page)
        self.table = torch.full((B, W), self.dummy, dtype=torch.int32, device=DEV)
        self.free = i32(np.random.default_rng(seed).permutation(pages))
        self.lens = i32([0] * B)
        self.cache = mk.minisgl_rope_table(mk.Rope(d // 2, kind="yarn", factor=4.0, original_positions=64), i32(range(W)))
        self.sm = d ** -0.5

    def store(self, extend, total, q, k, v):
        s = mk.minisgl_build_slots(self.lens, extend, self.table, self.free, self.page, self.dummy, total)
        q = mk.minisgl_rope_store_kv_fp8(self.pool, 0, q, k, v, s.positions, self.cache, s.out_loc,
                                         q_out=torch.empty_like(q))
        return s, q

    def finish(self, s):
        used = int(s.pages_used)
        assert used <= self.free.numel()
        self.free = self.free[used:].contiguous()
        self.lens = s.seq_lens.clone()

    def extend(self, s, extend, q, total):
        """All cached rows read back as a small bf16 pool, and attention over it."""
        table = torch.zeros_like(self.table)
        packed = mk.minisgl_build_slots(torch.zeros_like(s.seq_lens), s.seq_lens, table, i32(range(total)), 1, 0, total)
        wide = torch.zeros((2, 1, total, self.H, self.d), dtype=torch.bfloat16, device=DEV)
        mk.minisgl_load_kv_fp8(self.pool, 0, self.table, s.seq_lens, packed.q_offsets, total, wide[0, 0], wide[1, 0])
        return mk.minisgl_extend_attn(mk.KVPool(wide), 0, q, table, self.lens, extend, s.q_offsets, self.sm)


def test_prefill_in_chunks_then_decode_steps():
    """The operators as an engine runs them: two prefill chunks, then decode
    steps.  The cache holds the rotated rows within e4m3's half step (and what a
    block's growth adds), and attention is that over the pool's values."""
    B, Hq, H, d, page = 5, 16, 4, 128, 32
    eng = Engine(B, 288, 45, page, Hq, H, d, 7)
    rng = np.random.default_rng(7)
    kept = [[], []], [[] for _ in range(B)]
    rows_of = [[np.zeros((0, H, d))] * B, [np.zeros((0, H, d))] * B]
    cache = f64(eng.cache)

    def step(extend, seed):
        T = int(sum(extend))
        q, k, v = (kv_like((T, h, d), seed + i).to(DEV) for i, h in enumerate((Hq, H, H)))
        s, turned = eng.store(i32(extend), T, q, k, v)
        kr, _ = ref.rotate(f64(k), cache[s.positions.cpu().numpy()], False)
        at = 0
        for r, e in enumerate(extend):
            for i, x in enumerate((kr, f64(v))):
                rows_of[i][r] = np.concatenate([rows_of[i][r], x[at:at + e]])
            at += e
        return s, turned

    def check_cache(s):
        lens = s.seq_lens.tolist()
        assert lens == [len(x) for x in rows_of[0]]
        for i, vals in enumerate(pool_values(eng.pool)):
            for r, n in enumerate(lens):
                want, got = rows_of[i][r], vals[eng.table[r, :n].cpu().numpy()]
                top = np.array([np.abs(want[j // 16 * 16:j // 16 * 16 + 16]).max((0, 2)) for j in range(n)]).reshape(n, H, 1)
                # half a step; a subnormal's half steps at each growth of the scale, below 2^-9 * max / 224 in all;
                # and the rotation's fp32
                assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -9 * top / 224 + 1e-5).all()

    for chunk in range(2):
        extend = rng.integers(0, 100, B)
        extend[chunk] = 0
        s, q = step(extend, 100 * chunk)
        total = int(s.seq_lens.sum())
        o = f64(eng.extend(s, i32(extend), q, total))
        check_cache(s)
        k, v = pool_values(eng.pool)
        pt = eng.table.cpu().numpy()
        for i, (r, p) in enumerate(zip(np.repeat(np.arange(B), extend), s.positions.tolist())):
            # extend attention rounds its weights to bf16: 2^-8
            want, mag, top = fp4_ref.decode(f64(q[i:i + 1]), k, v, pt[r:r + 1, :p + 1], [p + 1], eng.sm)
            bound = fp4_ref.decode_bound(want, mag, top, np.abs(v).max(), p + 1, weight_step=2.0 ** -8)
            assert (np.abs(o[i:i + 1] - want) <= bound).all(), (chunk, i)
        eng.finish(s)
    for n in range(20):
        s, q = step([1] * B, 1000 + 10 * n)
        check_decode(eng.pool, q, eng.table, s.seq_lens.tolist(), eng.sm)
        check_cache(s)
        eng.finish(s)


def test_graph_of_a_decode_step_with_padding():
    """Slots, store and decode captured for a padded batch and replayed while
    the lengths advance in place; two graphs with workspaces of their own
    replayed at once on two streams."""
    B, Hq, H, d, page, steps = 6, 16, 8, 128, 16, 20
    made = []
    for _ in range(3):
        eng = Engine(B, 96, 60, page, Hq, H, d, 3)
        pre = i32([20, 0, 3, 40, 0, 0])
        q, k, v = (kv_like((63, h, d), h).to(DEV) for h in (Hq, H, H))
        s, _ = eng.store(pre, 63, q, k, v)
        eng.free = eng.free[int(s.pages_used):].contiguous()
        eng.lens = i32([20, 0, 3, 40, -1, -1])
        q, k, v = (kv_like((B, h, d), 50 + h).to(DEV) for h in (Hq, H, H))
        made.append((eng, i32([1] * B), q, k, v, mk.decode_workspace_fp8(B, Hq, eng.pool)))

    def step(x):
        eng, one, q, k, v, ws = x
        s, q = eng.store(one, B, q, k, v)
        o = mk.minisgl_decode_attn_fp8(eng.pool, 0, q, eng.table, s.seq_lens, eng.sm, workspace=ws)
        eng.lens[:4] += 1
        eng.free.copy_(torch.roll(eng.free, -4))  # pages never handed out twice in these steps
        k.mul_(1.25)  # scales grow
        return o

    want = [step(made[0]).clone() for _ in range(steps)]
    check_decode(made[0][0].pool, *decode_args_of(made[0][0], made[0]))
    graphs = []
    for x in made[1:]:
        eng = x[0]
        live = (eng.lens, eng.free, eng.table, eng.pool.data, eng.pool.scales, x[3])
        saved = [t.clone() for t in live]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(x)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = step(x)
        for t, y in zip(live, saved):
            t.copy_(y)
        graphs.append((g, o, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(steps):
        for g, _, st in graphs:
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for _, o, _ in graphs:
            assert torch.equal(o[:4], want[i][:4]), f"step {i}"


def decode_args_of(eng, x):
    """q, table, lengths and scale of a decode call over what the engine has cached."""
    return x[2], eng.table, [max(n, 0) for n in eng.lens.tolist()], eng.sm
