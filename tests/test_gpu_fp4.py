"""GPU tests of the 4-bit pool's calls against the plain 64-bit definitions in
tests/fp4_ref.py.  Slots, stored bytes and loaded values must be equal; decode
attention stays within bounds counted from its roundings (fp4_ref.decode_bound)."""
import math
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_kv_cache_row_gb300 as mk
from tests import fp4_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_row_gb300 import build
    build.build()
    assert torch.cuda.is_available()


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def pool_values(pool, layer=0):
    """float64 K and V [R, H, d] of a layer."""
    d, s = pool.data.cpu().numpy(), pool.scales.cpu().numpy()
    return (ref.values(d[0, layer], s[0, layer], pool.k_exp[layer]),
            ref.values(d[1, layer], s[1, layer], pool.v_exp[layer]))


# --------------------------------------------------------------------------- #
# slots
# --------------------------------------------------------------------------- #
def check_slots(cached, extend, width, page, total=None, free_short=0, dummy=10 ** 6, stride=None, seed=0,
                cap_pages=None):
    rng = np.random.default_rng(seed)
    B = len(cached)
    total = sum(max(e, 0) for e in extend) if total is None else total
    table = rng.integers(-9, -1, size=(B, width))
    for r, c in enumerate(cached):  # cached rows in pages of their own
        for j in range(min(max(c, 0), width)):
            table[r, j] = (500 + r * 1000 + j // page) * page + j % page
    need = sum(max(0, -(-min(c + max(e, 0), width) // page) - -(-c // page))
               for c, e in zip(cached, extend) if c >= 0)
    free = rng.permutation(need + 5)[:max(0, need + 5 - free_short)] if cap_pages is None else \
        rng.permutation(cap_pages)
    want = ref.build_slots(cached, extend, table, free, page, dummy, total)
    stride = stride or width
    buf = torch.full((B, stride), -77, dtype=torch.int32, device=DEV)
    pt = buf[:, :width]
    pt.copy_(i32(table))
    out = mk.Slots(*(torch.full((n + 3,), -7, dtype=torch.int32, device=DEV)[:n]
                     for n in (total, total, B + 1, B, 1)))
    mk.minisgl_build_slots(i32(cached), i32(extend), pt, i32(free), page, dummy, total, out=out)
    torch.cuda.synchronize()
    for got, w, nm in zip((pt,) + out[:4], want[:5], ("page_table", "out_loc", "positions", "q_offsets", "seq_lens")):
        assert np.array_equal(got.cpu().numpy(), w), nm
    assert int(out.pages_used) == want[5]
    if stride > width:
        assert bool((buf[:, width:] == -77).all()), "wrote past the table's width"
    return want


@pytest.mark.parametrize("page", [1, 7, 16, 64])
@pytest.mark.parametrize("B", [1, 5, 33, 700])
def test_slots_random(B, page):
    rng = np.random.default_rng(B * 100 + page)
    cached = rng.integers(0, 100, B)
    extend = rng.integers(0, 60, B)
    cached[rng.random(B) < 0.2] = 0
    extend[rng.random(B) < 0.2] = 0
    pad = rng.random(B) < 0.2
    cached[pad], extend[pad] = -1, 1
    check_slots(cached.tolist(), extend.tolist(), 160, page, seed=B, stride=167)


def test_slots_decode_step_of_the_largest_batch():
    check_slots([63 + r % 70 for r in range(4096)], [1] * 4096, 160, 64, seed=3)


def test_slots_largest_batch_ragged():
    rng = np.random.default_rng(8)
    check_slots(rng.integers(-1, 40, 4096).tolist(), rng.integers(0, 9, 4096).tolist(), 64, 16, seed=4)


def test_slots_page_borders():
    c = [0, 15, 16, 17, 31, 32, 0, 1, 16, 48]
    check_slots(c, [16, 1, 1, 15, 1, 16, 0, 0, 0, 16], 64, 16)


def test_slots_out_of_pages():
    """Four pages too few: the last tokens are on the dummy row, the count says what was needed."""
    want = check_slots([5, 0, 9], [40, 33, 20], 64, 8, free_short=9)
    assert (want[1] == 10 ** 6).sum() > 0 and want[5] == 12
    check_slots([5, 0, 9], [40, 33, 20], 64, 8, cap_pages=0)


@pytest.mark.parametrize("dummy", [0, 1, 3, 99])
def test_slots_after_running_out_of_pages(dummy):
    """A request that goes on after its page lay past the free pages: the rest
    of that page stays on the dummy row (the first of a page, inside one, the
    last of one whose next row is another request's, past the pool), and the
    page behind it is a new one."""
    D = dummy
    table = torch.full((2, 16), -1, dtype=torch.int32, device=DEV)
    steps = [([0, 0], [2, 6], [1], [4, 5] + [D] * 6, 3), ([2, 6], [1, 3], [2], [6, D, D, 8], 1),
             ([3, 9], [1, 1], [5], [7, 9], 0), ([4, 10], [2, 1], [5], [20, 21, 10], 1)]
    for cached, extend, free, loc, used in steps:
        s = mk.minisgl_build_slots(i32(cached), i32(extend), table, i32(free), 4, D, sum(extend))
        assert s.out_loc.tolist() == loc and s.pages_used.item() == used
    assert table.tolist() == [[4, 5, 6, 7, 20, 21] + [-1] * 10, [D] * 8 + [8, 9, 10] + [-1] * 5]


def test_slots_tail_width_and_short_total():
    check_slots([3, 0], [4, 5], 32, 4, total=50)             # captured for 50 tokens
    check_slots([30, 0, 40], [10, 5, 3], 32, 4)              # past the table's width
    check_slots([3, 0, 8], [4, 5, 6], 32, 4, total=7)        # fewer rows than tokens
    check_slots([3, 0, 8], [4, 5, 6], 32, 4, total=0)
    check_slots([3, -1, -1, 8], [0, 4, -3, -6], 32, 4, total=6)


def test_slots_empty_batch_and_saturating_lengths():
    z = i32([])
    s = mk.minisgl_build_slots(z, z, torch.zeros((0, 32), dtype=torch.int32, device=DEV), i32([1]), 4, 9, 3)
    assert s.out_loc.tolist() == [9, 9, 9] and s.positions.tolist() == [0, 0, 0]
    assert s.q_offsets.tolist() == [0] and s.pages_used.tolist() == [0]
    big = 2 ** 31 - 1  # lengths that no batch has: nothing overflows, nothing is written out of place
    pt = torch.full((3, 32), -1, dtype=torch.int32, device=DEV)
    s = mk.minisgl_build_slots(i32([0, big, 5]), i32([big, big, big]), pt, i32(range(40)), 4, 9, 40)
    assert pt[0].tolist() == list(range(32)) and s.out_loc[32:].tolist() == [9] * 8
    assert s.q_offsets.tolist() == [0] + [2 ** 30] * 3 and s.seq_lens.tolist() == [32, 32, 32]
    assert bool((pt[1:] == -1).all())


# --------------------------------------------------------------------------- #
# store and load
# --------------------------------------------------------------------------- #
def kv_like(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(0.5 * torch.randn(shape[-2:], generator=g)) * scale
    return x.to(torch.bfloat16)


def check_store(pool, layer, k, v, out_loc, exact_codes=True):
    """Stored bytes equal the definition's, all other bytes are unchanged."""
    want_d, want_s = pool.data.cpu().numpy().copy(), pool.scales.cpu().numpy().copy()
    for i, (x, e) in enumerate(((k, pool.k_exp[layer]), (v, pool.v_exp[layer]))):
        codes, sb = ref.quantise(ref.bf16_to_f64(x), e)
        want_d[i, layer][out_loc] = ref.pack(codes)
        want_s[i, layer][out_loc] = sb
    mk.minisgl_store_kv_fp4(pool, layer, k, v, i32(out_loc))
    torch.cuda.synchronize()
    got_d, got_s = pool.data.cpu().numpy(), pool.scales.cpu().numpy()
    assert np.array_equal(got_s, want_s), "scales"
    if exact_codes:
        assert np.array_equal(got_d, want_d), "elements"


@pytest.mark.parametrize("H,d", [(1, 64), (2, 64), (3, 128), (5, 64), (8, 128)])
@pytest.mark.parametrize("n", [1, 2, 37, 1000])
def test_store_bytes(H, d, n):
    pool = mk.KVPoolFP4.zeros(2, n + 40, H, d, k_exp=[-1, 3], v_exp=-2)
    pool.data.fill_(0x5A)
    pool.scales.fill_(0x33)
    rows = np.random.default_rng(n).permutation(n + 40)[:n]
    check_store(pool, 1, kv_like((n, H, d), n).to(DEV), kv_like((n, H, d), n + 1, 0.1).to(DEV), rows)


def test_store_strided_rows_and_page_first_pool():
    """K and V cut out of one projection's output, rows every other token, and a
    pool whose rows hold all layers (pages outermost)."""
    L, R, H, d, n = 3, 60, 4, 128, 20
    data = torch.zeros((2, R, L, H, d // 2), dtype=torch.uint8, device=DEV).transpose(1, 2)
    scales = torch.zeros((2, R, L, H, d // 16), dtype=torch.uint8, device=DEV).transpose(1, 2)
    pool = mk.KVPoolFP4(data, scales.view(torch.float8_e4m3fn), k_exp=0, v_exp=1)
    qkv = kv_like((2 * n, 3 * H, d), 5).to(DEV)
    check_store(pool, 1, qkv[::2, H:2 * H], qkv[1::2, 2 * H:], np.random.default_rng(1).permutation(R)[:n])


def test_store_every_largest_value():
    """A block for every finite bf16 as its largest element, the others spread below it."""
    amax = torch.arange(0, 0x7F80, dtype=torch.int16)
    amax = torch.cat([amax, amax.new_zeros((-len(amax)) % 8)]).view(torch.bfloat16)
    rng = np.random.default_rng(2)
    frac = torch.from_numpy(rng.uniform(-1, 1, size=(len(amax), 16)))
    x = (amax.double()[:, None] * frac).to(torch.bfloat16)
    x = torch.where(x.double().abs() <= amax.double()[:, None], x, torch.zeros_like(x))
    x[torch.arange(len(amax)), torch.from_numpy(rng.integers(0, 16, len(amax)))] = amax
    x = x.reshape(-1, 1, 128)
    for e in (-64, -3, 0, 64):
        pool = mk.KVPoolFP4.zeros(1, x.shape[0], 1, 128, k_exp=e, v_exp=-e)
        check_store(pool, 0, x.to(DEV), -x.to(DEV), np.arange(x.shape[0]))


def test_store_ties():
    """Elements exactly on the borders between e2m1 values, and bf16 neighbours of them, for every scale."""
    s = torch.from_numpy(ref.E4M3[1:]).double()
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    x = torch.zeros((len(s), 64), dtype=torch.bfloat16)
    for b in range(4):  # each block: its largest is 6 s, then borders and neighbours
        x[:, 16 * b] = (6 * s).to(torch.bfloat16)
        bits = (border[None] * s[:, None]).to(torch.bfloat16).view(torch.int16)
        x[:, 16 * b + 1:16 * b + 8] = (bits + (0, 1, -1, 0)[b]).view(torch.bfloat16)
        x[:, 16 * b + 8:16 * b + 15] = -((bits + (0, -1, 1, 2)[b]).view(torch.bfloat16))
    x = x[:, None, :]
    pool = mk.KVPoolFP4.zeros(1, len(s), 1, 64)
    check_store(pool, 0, x.to(DEV), -x.to(DEV), np.arange(len(s)))


def test_store_nan_and_infinity():
    x = kv_like((6, 1, 64), 3)
    x[1, 0, 5] = math.nan
    x[2, 0, 17] = math.inf
    x[3, 0, 20], x[3, 0, 21], x[3, 0, 22] = -math.inf, math.inf, 2.0
    x[4, 0, 40], x[4, 0, 41] = math.inf, -math.nan
    x[5] = 0
    pool = mk.KVPoolFP4.zeros(1, 6, 1, 64)
    check_store(pool, 0, x.to(DEV), x.to(DEV), np.arange(6), exact_codes=False)
    k, _ = pool_values(pool)
    want = ref.values(ref.pack(ref.quantise(ref.bf16_to_f64(x), 0)[0]), ref.quantise(ref.bf16_to_f64(x), 0)[1], 0)
    assert np.array_equal(k[:, 0], want[:, 0], equal_nan=True)
    assert np.isnan(k[1, 0, :16]).all() and np.isfinite(k[1, 0, 16:]).all()
    assert k[2, 0, 17] == 2688 and k[3, 0, 20] == -2688 and np.isnan(k[4, 0, 32:48]).all()
    assert (k[5] == 0).all()


def test_store_clamps_rows_and_does_nothing_for_no_tokens():
    pool = mk.KVPoolFP4.zeros(1, 4, 2, 64)
    k = kv_like((3, 2, 64), 1).to(DEV)
    mk.minisgl_store_kv_fp4(pool, 0, k, k, i32([-5, 1, 99]))
    kk, _ = pool_values(pool)
    assert (kk[2] == 0).all() and (kk[0] != 0).any() and (kk[3] != 0).any()
    mk.minisgl_store_kv_fp4(pool, 0, k[:0], k[:0], i32([]))
    torch.cuda.synchronize()


def random_pool(L, R, H, d, seed, k_exp=-2, v_exp=-1, lo=0x18, hi=0x48):
    """A pool of random elements and scales from 2^-4 to 2^2; the last row is NaN."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    pool = mk.KVPoolFP4.zeros(L, R, H, d, k_exp=k_exp, v_exp=v_exp)
    pool.data.random_(0, 256, generator=g)
    pool.scales.random_(lo, hi, generator=g)
    pool.scales[:, :, R - 1] = 0x7F
    return pool


@pytest.mark.parametrize("H,d", [(1, 64), (3, 64), (8, 128), (5, 128)])
def test_load_rows(H, d):
    rng = np.random.default_rng(H)
    R, lens = 500, [0, 1, 70, 33, 0, 64, 5]
    pool = random_pool(2, R, H, d, H, k_exp=[0, 5], v_exp=[1, -7], lo=0, hi=256)
    W = 64  # request 2 is longer than the table is wide
    pt = np.full((len(lens), W), R - 1)
    for r, n in enumerate(lens):
        pt[r, :min(n, W)] = rng.permutation(R - 1)[:min(n, W)]
    gaps = [2, 0, 3, 1, 0, 2, 4]  # rows between the requests
    off = np.concatenate([[3], 3 + np.cumsum(np.array(lens) + gaps)])
    total = int(off[-1]) - 6  # the last rows do not fit
    k_out = torch.full((total, H * d + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    v_out = torch.full((total, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
    mk.minisgl_load_kv_fp4(pool, 1, i32(pt), i32(lens), i32(off), total, k_out[:, :H * d], v_out)
    torch.cuda.synchronize()
    kv = pool_values(pool, 1)
    for got, x in ((k_out[:, :H * d].reshape(total, H, d), kv[0]), (v_out, kv[1])):
        want = np.full((total, H, d), 7.0)
        for r, n in enumerate(lens):
            for j in range(min(n, W)):
                if off[r] + j < total:
                    want[off[r] + j] = x[pt[r, j]]
        assert np.array_equal(got.double().cpu().numpy(), want, equal_nan=True)
    assert bool((k_out[:, H * d:] == 7).all())


def test_load_many_short_requests():
    R, H, d, B = 300, 2, 64, 4096
    pool = random_pool(1, R, H, d, 9)
    lens = np.random.default_rng(0).integers(0, 3, B)
    lens[100:900] = 0
    pt = np.random.default_rng(1).integers(0, R - 1, (B, 3))
    off = np.concatenate([[0], np.cumsum(lens)])
    k, v = mk.minisgl_load_kv_fp4(pool, 0, i32(pt), i32(lens), i32(off), int(off[-1]))
    rows = np.concatenate([pt[r, :n] for r, n in enumerate(lens)])
    kv = pool_values(pool)
    assert np.array_equal(k.double().cpu().numpy(), kv[0][rows])
    assert np.array_equal(v.double().cpu().numpy(), kv[1][rows])


@pytest.mark.parametrize("H,d", [(33, 128), (40, 128), (130, 64)])
def test_rows_wider_than_a_block_of_threads(H, d):
    """Store, load and decode with more than 512 blocks of 16 in a token's row."""
    n = 40
    pool = mk.KVPoolFP4.zeros(1, 64, H, d, k_exp=-2, v_exp=-2)
    at = np.random.default_rng(H).permutation(64)[:n]
    k, v = kv_like((n, H, d), H).to(DEV), kv_like((n, H, d), H + 1).to(DEV)
    check_store(pool, 0, k, v, at)
    kv = pool_values(pool)
    for got, want in zip(mk.minisgl_load_kv_fp4(pool, 0, i32(at[None]), i32([n]), i32([0, n]), n), kv):
        assert np.array_equal(got.double().cpu().numpy(), want[at])
    check_decode(pool, kv_like((1, H, d), 5).to(DEV), at[None], [n])


def test_load_every_value():
    """Every element under every scale, at exponents whose values bf16 holds."""
    R = 256
    for e in (-64, 0, 64):
        pool = mk.KVPoolFP4.zeros(1, R, 1, 64, k_exp=e, v_exp=e)
        pool.data[:] = torch.arange(32, dtype=torch.uint8, device=DEV) * 8 + 5
        pool.data[0, 0, :, 0, :16] = torch.arange(16, dtype=torch.uint8, device=DEV) * 17
        pool.scales[:] = torch.arange(R, dtype=torch.uint8, device=DEV)[None, None, :, None, None]
        k, v = mk.minisgl_load_kv_fp4(pool, 0, i32([range(R)]), i32([R]), i32([0, R]), R)
        kv = pool_values(pool)
        assert np.array_equal(k.double().cpu().numpy(), kv[0], equal_nan=True)
        assert np.array_equal(v.double().cpu().numpy(), kv[1], equal_nan=True)


# --------------------------------------------------------------------------- #
# decode
# --------------------------------------------------------------------------- #
def make_decode(Hq, Hkv, d, lens, R, seed, page=1, q_scale=1.0, **kw):
    pool = random_pool(1, R, Hkv, d, seed, **kw)
    rng = np.random.default_rng(seed)
    W = max(1, -(-max(lens) // 32) * 32)
    pt = np.full((len(lens), W), R - 1)
    pages = (R - 1) // page
    for r, n in enumerate(lens):
        mine = rng.permutation(pages)[:-(-n // page)]
        assert len(mine) * page >= n
        j = np.arange(n)
        pt[r, :n] = mine[j // page] * page + j % page
    q = (torch.from_numpy(rng.normal(size=(len(lens), Hq, d))) * q_scale).to(torch.bfloat16).to(DEV)
    return pool, q, pt


def check_decode(pool, q, pt, lens, sm_scale=None, table=None, **kw):
    sm = 1 / math.sqrt(q.shape[2]) if sm_scale is None else sm_scale
    o = mk.minisgl_decode_attn_fp4(pool, 0, q, i32(pt) if table is None else table, i32(lens), sm, **kw)
    torch.cuda.synchronize()
    k, v = pool_values(pool)
    want, mag, top = ref.decode(ref.bf16_to_f64(q), k, v, pt, lens, sm)
    got = o.double().cpu().numpy()
    assert np.isfinite(want).all()
    fine = np.isfinite(v)
    bound = ref.decode_bound(want, mag, top, np.abs(v[fine]).max(), max(lens))
    err = np.abs(got - want)
    assert np.isfinite(got).all() and (err <= bound).all(), (float((err / bound).max()), float(err.max()))
    return o


SHAPES = [(8, 2, 64), (16, 8, 128), (4, 4, 128), (32, 2, 128), (16, 1, 64), (24, 8, 64), (9, 1, 128), (6, 3, 64),
          (5, 5, 128), (18, 9, 64), (12, 12, 128), (34, 17, 64), (112, 16, 128), (22, 2, 64)]


@pytest.mark.parametrize("Hq,Hkv,d", SHAPES, ids=["%d-%d-%d" % s for s in SHAPES])
def test_decode_head_layouts(Hq, Hkv, d):
    lens = [0, 1, 2, 31, 32, 33, 64, 100, 257, 0, 400]
    pool, q, pt = make_decode(Hq, Hkv, d, lens, 700, Hq + Hkv + d)
    check_decode(pool, q, pt, lens)


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 64), (16, 8, 128), (32, 2, 128), (11, 11, 128), (7, 7, 64), (20, 10, 64)])
def test_decode_short_tables(Hq, Hkv, d):
    """Tables narrow enough for every request to be left whole."""
    for lens in ([0, 1, 31, 32, 33, 100, 128, 0], [5], [0], [1] * 40 + [32] * 3):
        pool, q, pt = make_decode(Hq, Hkv, d, lens, 200, Hq + Hkv + d)
        check_decode(pool, q, pt, lens)


@pytest.mark.parametrize("B", [149, 152, 153, 302, 304, 305])
@pytest.mark.parametrize("width", [160, 256, 288, 2048])
def test_decode_batches_near_the_number_of_groups(B, width):
    """One request as long as the table is wide, empty ones and short ones, at
    batches around one and two groups of warps on each of 152 SMs."""
    lens = [(0, 1, 30, 33, 64, 7)[r % 6] for r in range(B)]
    lens[B // 2] = width
    pool, q, pt = make_decode(16, 8, 128, lens, 2100, B + width)
    assert pt.shape[1] == width
    check_decode(pool, q, pt, lens)


@pytest.mark.parametrize("H,d", [(8, 128), (2, 128), (4, 64), (16, 128), (3, 64)])
def test_scale_rows_that_start_anywhere(H, d):
    """Scale rows only d/16-byte aligned (a slice of wider rows), elements in
    rows of all layers (pages outermost): store, load and decode."""
    L, R, SB = 2, 150, d // 16
    data = torch.zeros((2, R, L, H, d // 2), dtype=torch.uint8, device=DEV).transpose(1, 2)
    scales = torch.zeros((2, L, R, H + 1, SB), dtype=torch.uint8, device=DEV)[:, :, :, 1:]
    pool = mk.KVPoolFP4(data, scales, k_exp=[0, -2], v_exp=[0, -1])
    n, lens = 130, [50, 80]
    rows = np.random.default_rng(1).permutation(R)[:n]
    check_store(pool, 1, kv_like((n, H, d), 1).to(DEV), kv_like((n, H, d), 2).to(DEV), rows)
    pt = np.zeros((2, 96), dtype=int)
    pt[0, :50], pt[1, :80] = rows[:50], rows[50:]
    kv = pool_values(pool, 1)
    k, v = mk.minisgl_load_kv_fp4(pool, 1, i32(pt), i32(lens), i32([0, 50, 130]), n)
    assert np.array_equal(k.double().cpu().numpy(), kv[0][rows])
    assert np.array_equal(v.double().cpu().numpy(), kv[1][rows])
    q = kv_like((2, 2 * H, d), 3).to(DEV)
    for split in (0, 32):
        o = mk.minisgl_decode_attn_fp4(pool, 1, q, i32(pt), i32(lens), d ** -0.5, split_tokens=split)
        want, mag, top = ref.decode(ref.bf16_to_f64(q), kv[0], kv[1], pt, lens, d ** -0.5)
        bound = ref.decode_bound(want, mag, top, np.abs(kv[1]).max(), 80)
        assert (np.abs(o.double().cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("slots", [0, 1, 4], ids=["packed", "one-more", "aligned"])
@pytest.mark.parametrize("H,d", [(11, 128), (15, 64), (15, 128), (17, 128), (25, 64), (30, 64), (57, 128)])
def test_decode_short_last_head_block(H, d, slots):
    """Head counts whose last block has fewer heads than the others, up to the
    pool's last row, with rows of scales that end with the pool's memory or
    have room for more heads behind them."""
    R, lens = 150, [150, 40]
    room = -(-H // slots) * slots + (slots == 1) if slots else H
    data = torch.zeros((2, 1, R, H, d // 2), dtype=torch.uint8, device=DEV)
    scales = torch.full((2, 1, R, room, d // 16), 0x7F, dtype=torch.uint8, device=DEV)[:, :, :, :H]
    pool = mk.KVPoolFP4(data, scales, k_exp=-2, v_exp=-1)
    pool.data.random_(0, 256)
    pool.scales.random_(0x18, 0x48)
    pt = np.zeros((2, 160), dtype=int)
    pt[0, :150] = np.random.default_rng(H).permutation(R)
    pt[1, :40] = R - 1 - np.arange(40)
    q = kv_like((2, 2 * H, d), 3).to(DEV)
    check_decode(pool, q, pt, lens)
    check_decode(pool, q, pt, lens, split_tokens=32)


@pytest.mark.parametrize("split", [1, 32, 48, 100, 10 ** 6])
@pytest.mark.parametrize("max_splits", [2, 5, 64, 256])
def test_decode_split_counts(split, max_splits):
    lens = [900, 1, 65, 0, 333]
    pool, q, pt = make_decode(16, 4, 128, lens, 1000, 11)
    check_decode(pool, q, pt, lens, split_tokens=split, max_splits=max_splits)


@pytest.mark.parametrize("Hq,Hkv,d,page,lens", [
    (32, 8, 128, 64, [1500, 3000, 64, 2049]),
    (64, 8, 128, 16, [5000]),
    (16, 16, 64, 1, [4097, 4095]),
    (8, 1, 128, 64, [20000, 3])], ids=["pages64", "one-request", "mha", "mqa-long"])
def test_decode_long(Hq, Hkv, d, page, lens):
    pool, q, pt = make_decode(Hq, Hkv, d, lens, 20500 // 64 * 64 + 1, 21, page=page)
    check_decode(pool, q, pt, lens)


def test_decode_many_requests():
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 40, 4096).tolist()
    pool, q, pt = make_decode(4, 2, 64, lens, 300, 5)
    check_decode(pool, q, pt, lens)


@pytest.mark.parametrize("Hq,Hkv,d", [(32, 2, 64), (16, 8, 128)])
def test_decode_split_into_many_rows(Hq, Hkv, d):
    """More query rows than one wave of the merge's wide form."""
    lens = [(r * 37) % 190 for r in range(200)]
    pool, q, pt = make_decode(Hq, Hkv, d, lens, 300, 29)
    check_decode(pool, q, pt, lens, split_tokens=32)
    check_decode(pool, q, pt, lens, split_tokens=32, max_splits=3)


def test_decode_sharp_scores():
    """Scores spread over hundreds, rising and falling along the context, so
    that the running reference moves many times, and a negative scale."""
    lens = [700, 129, 1]
    pool, q, pt = make_decode(8, 2, 128, lens, 800, 31, q_scale=8.0)
    k, _ = pool_values(pool)
    for r, n in enumerate(lens):  # order request r's rows by head 0's score
        s = k[pt[r, :n], 0] @ ref.bf16_to_f64(q)[r, 0]
        pt[r, :n] = pt[r, :n][np.argsort(s if r % 2 == 0 else -s)]
    check_decode(pool, q, pt, lens)
    check_decode(pool, q, pt, lens, sm_scale=-0.05)
    check_decode(pool, q, pt, lens, sm_scale=0.0)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("power", [16, 23, 27, 31, 60, 112])
def test_decode_scores_of_any_size(power, sign):
    """Equal keys with scores from 2^20 to near fp32's largest: equal weights,
    so the mean of V, however coarse the scores' last place is."""
    lens = [1, 5, 33, 120]
    pool, q, pt = make_decode(8, 2, 64, lens, 200, 47)
    pool.data[0] = pool.data[0, :, :1] & 0x77  # one row of positive elements
    pool.scales[0] = pool.scales[0, :, :1]
    q = (q.abs() * sign * 2.0 ** power).contiguous()
    k, v = pool_values(pool)
    o = mk.minisgl_decode_attn_fp4(pool, 0, q, i32(pt), i32(lens), 0.125).double().cpu().numpy()
    for r, n in enumerate(lens):
        rows = v[pt[r, :n]].repeat(4, axis=1)
        want, mag = rows.mean(0), np.abs(rows).mean(0)
        bound = ref.decode_bound(want, mag, np.zeros(8), np.nanmax(np.abs(v)), n)
        assert (np.abs(o[r] - want) <= bound).all(), r
    # split: V is one row too
    pool.data[1] = pool.data[1, :, :1]
    pool.scales[1] = pool.scales[1, :, :1]
    pt = np.zeros((1, 2016))
    want = pool_values(pool)[1][0].repeat(4, axis=0)
    o = mk.minisgl_decode_attn_fp4(pool, 0, q[:1], i32(pt), i32([2000]), np.float32(0.125)).double().cpu().numpy()[0]
    assert (np.abs(o - want) <= ref.decode_bound(want, np.abs(want), np.zeros(8), np.abs(want).max(), 2000)).all()


@pytest.mark.parametrize("power", [-120, -40, 40, 100])
def test_decode_query_and_pool_ranges(power):
    """q from far below to far above fp16's range against the opposite scale
    and pool exponents."""
    lens = [200, 40]
    e = max(-64, min(64, -power // 2))
    pool, q, pt = make_decode(8, 4, 64, lens, 300, 41, q_scale=2.0 ** power, k_exp=e, v_exp=-60)
    q[0, 3] = 0  # a head of zeros: the mean of V
    check_decode(pool, q, pt, lens, sm_scale=2.0 ** (-power - e) / 8)


def test_decode_small_query_elements_count():
    """Elements 2^20 times smaller than the head's largest, against keys that
    are zero where the large ones are."""
    lens = [90]
    pool, q, pt = make_decode(4, 2, 128, lens, 100, 43)
    pool.scales[0, 0, :99, :, 0] = 0  # channels 0..15 of K are zero
    q[:, :, 0] = 2.0 ** 20
    check_decode(pool, q, pt, lens)


def test_decode_zero_and_full_range_scales():
    """Scales from 0 and 2^-9 to 448 next to one another."""
    lens = [300, 77]
    pool, q, pt = make_decode(16, 2, 128, lens, 400, 51, lo=0, hi=0x7F, k_exp=-10, v_exp=3)
    check_decode(pool, q, pt, lens)


def test_decode_nan_stays_in_its_head():
    lens = [100, 50]
    pool, q, pt = make_decode(8, 4, 64, lens, 200, 61)
    row = next(int(x) for x in pt[0, 30:100] if x not in pt[1, :50])
    clean = mk.minisgl_decode_attn_fp4(pool, 0, q, i32(pt), i32(lens), 0.125)
    pool.scales[0, 0, row, 2, 1] = 0x7F   # K of head 2: its scores
    pool.scales[1, 0, row, 1, 3] = 0x7F   # V of head 1: channels 48..63
    o = mk.minisgl_decode_attn_fp4(pool, 0, q, i32(pt), i32(lens), 0.125)
    bad = torch.zeros_like(o, dtype=torch.bool)
    bad[0, 4:6] = True
    bad[0, 2:4, 48:] = True
    assert torch.equal(torch.isnan(o), bad)
    assert torch.equal(o[~bad], clean[~bad])


def test_decode_table_stride_workspace_and_out():
    """A table cut out of a wider one, a workspace full of NaN, a given out."""
    lens = [600, 3, 250]
    pool, q, pt = make_decode(32, 8, 128, lens, 700, 71)
    wide = torch.full((3, pt.shape[1] + 40), 10 ** 9, dtype=torch.int32, device=DEV)
    wide[:, :pt.shape[1]] = i32(pt)
    ws = mk.decode_workspace_fp4(3, 32, pool)
    ws.fill_(0xFF)
    out = torch.full_like(q, math.nan)
    o = check_decode(pool, q, pt, lens, table=wide[:, :pt.shape[1]], workspace=ws, out=out)
    assert o is out
    again = mk.minisgl_decode_attn_fp4(pool, 0, q, i32(pt), i32(lens), 1 / math.sqrt(128))
    assert torch.equal(o, again)  # no atomics: the same bits every time


def test_decode_lengths_past_the_table_are_clamped():
    pool, q, pt = make_decode(8, 2, 64, [64, 32], 100, 81)
    pt[1, 32:] = pt[1, :32]
    a = mk.minisgl_decode_attn_fp4(pool, 0, q, i32(pt), i32([10 ** 6, -4]), 0.125)
    b = mk.minisgl_decode_attn_fp4(pool, 0, q, i32(pt), i32([64, 0]), 0.125)
    assert torch.equal(a, b) and bool((a[1] == 0).all())


def test_rows_past_32_bit_offsets():
    """A pool whose last rows lie more than 2^32 bytes behind its base."""
    H, d = 8, 128
    R = (1 << 32) // (H * d // 2) + 3000
    pool = mk.KVPoolFP4(torch.empty((2, 1, R, H, d // 2), dtype=torch.uint8, device=DEV),
                        torch.empty((2, 1, R, H, d // 16), dtype=torch.uint8, device=DEV), k_exp=-2, v_exp=-2)
    n = 500
    rows = R - 1 - np.random.default_rng(0).permutation(2500)[:n]
    k, v = kv_like((n, H, d), 1).to(DEV), kv_like((n, H, d), 2).to(DEV)
    mk.minisgl_store_kv_fp4(pool, 0, k, v, i32(rows))
    small = mk.KVPoolFP4.zeros(1, n, H, d, k_exp=-2, v_exp=-2)
    mk.minisgl_store_kv_fp4(small, 0, k, v, i32(range(n)))
    q = kv_like((1, 16, d), 3).to(DEV)
    a = mk.minisgl_decode_attn_fp4(pool, 0, q, i32(rows[None]), i32([n]), 0.1)
    b = mk.minisgl_decode_attn_fp4(small, 0, q, i32([range(n)]), i32([n]), 0.1)
    assert torch.equal(a, b)
    la = mk.minisgl_load_kv_fp4(pool, 0, i32(rows[None]), i32([n]), i32([0, n]), n)
    lb = mk.minisgl_load_kv_fp4(small, 0, i32([range(n)]), i32([n]), i32([0, n]), n)
    assert torch.equal(la[0], lb[0]) and torch.equal(la[1], lb[1])


# --------------------------------------------------------------------------- #
# streams, graphs, and the operators together
# --------------------------------------------------------------------------- #
def test_calls_on_a_named_stream():
    """Work queued on another stream than the current one, with the call's own
    workspace and output, while the current stream reuses freed memory."""
    lens = [800, 500]
    pool, q, pt = make_decode(32, 8, 128, lens, 900, 91)
    table, sl = i32(pt), i32(lens)
    want = mk.minisgl_decode_attn_fp4(pool, 0, q, table, sl, 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(20):
        outs.append(mk.minisgl_decode_attn_fp4(pool, 0, q, table, sl, 0.1, stream=side))
        torch.full((1 << 22,), 255, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_loaded_rows_into_a_bf16_pool():
    """Slots, load and minisgl_store_kv in a captured chain whose buffers are
    used again by every round: each round's rows arrive, not the last one's."""
    H, d, n, rounds = 8, 128, 2000, 6
    pools = [random_pool(1, n + 1, H, d, 100 + i) for i in range(rounds)]
    bf = [torch.zeros((2, 1, n + 1, H, d), dtype=torch.bfloat16, device=DEV) for _ in range(rounds)]
    table, none, some, free = i32([range(n)]), i32([0]), i32([n]), i32(range(n))
    own = torch.zeros((1, n), dtype=torch.int32, device=DEV)
    k, v = (torch.zeros((n, H, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    out = mk.Slots.empty(1, n)

    def chain():
        for i in range(rounds):
            s = mk.minisgl_build_slots(none, some, own, torch.roll(free, i * 7), 1, n, n, out=out)
            mk.minisgl_load_kv_fp4(pools[i], 0, table, s.seq_lens, s.q_offsets, n, k, v)
            mk.minisgl_store_kv(mk.KVPool(bf[i]), 0, k, v, s.out_loc)
    chain()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain()
    for t in bf:
        t.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for i in range(rounds):
        rows = np.roll(np.arange(n), i * 7)
        for got, want in zip(bf[i][:, 0, rows], pool_values(pools[i])):
            assert np.array_equal(got.double().cpu().numpy(), want[:n])


FIRST_USE = """
import torch, paged_kv_cache_row_gb300 as mk
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
H, d, n = 2, 64, 70
pool = mk.KVPoolFP4.zeros(1, 81, H, d, 4, k_exp=-2, v_exp=-2)
kv = [torch.randn(n, H, d, device="cuda").to(torch.bfloat16) for _ in range(2)]
q = torch.randn(1, 4, d, device="cuda").to(torch.bfloat16)
table, free, none, some = i32([[0] * 96]), i32(list(range(20))), i32([0]), i32([n])
def step():
    s = mk.minisgl_build_slots(none, some, table, free, 4, 80, n)
    mk.minisgl_store_kv_fp4(pool, 0, *kv, s.out_loc)
    k, v = mk.minisgl_load_kv_fp4(pool, 0, table, s.seq_lens, s.q_offsets, n)
    return k, v, mk.minisgl_decode_attn_fp4(pool, 0, q, table, s.seq_lens, 0.125)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = step()
g.replay()
torch.cuda.synchronize()
got = [x.clone() for x in got]
assert all(torch.equal(a, b) for a, b in zip(got, step())) and got[2].abs().max() > 0
print("same")
"""


def test_first_use_may_be_captured():
    """A new process whose first calls are captured, with no call before them."""
    r = subprocess.run([sys.executable, "-c", FIRST_USE], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_binding_refusals():
    lens = [80, 50]
    pool, q, pt = make_decode(32, 8, 128, lens, 90, 91)
    table, sl = i32(pt), i32(lens)
    with pytest.raises(mk.MinisglError, match="q must be"):
        mk.minisgl_decode_attn_fp4(pool, 0, q[:, :, ::2], table, sl, 0.1)
    with pytest.raises(mk.MinisglError, match="out must be"):
        mk.minisgl_decode_attn_fp4(pool, 0, q, table, sl, 0.1, out=torch.empty_like(q[:1]))
    with pytest.raises(mk.MinisglError, match="layer"):
        mk.minisgl_decode_attn_fp4(pool, 1, q, table, sl, 0.1)
    with pytest.raises(mk.MinisglError, match="workspace"):
        mk.minisgl_decode_attn_fp4(pool, 0, q, table, sl, 0.1, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(mk.MinisglError, match="k must be"):
        mk.minisgl_store_kv_fp4(pool, 0, q, q, sl)
    with pytest.raises(mk.MinisglError, match="offsets"):
        mk.minisgl_load_kv_fp4(pool, 0, table, sl, sl, 4)
    with pytest.raises(mk.MinisglError, match="k_exp"):
        mk.KVPoolFP4(pool.data, pool.scales, k_exp=[1, 2])
    with pytest.raises(mk.MinisglError, match="extend_lens"):
        mk.minisgl_build_slots(sl, sl[:1], table, sl, 4, 0, 2)
    with pytest.raises(mk.MinisglError, match="overlaps an input"):
        s = mk.Slots.empty(2, 2)
        mk.minisgl_build_slots(sl, sl.clone(), table, sl, 4, 0, 2, out=s._replace(seq_lens=sl))


def test_outputs_are_filled_where_torch_fills_new_memory():
    """With deterministic algorithms torch fills new tensors with NaN; rows of
    a load that no request fills show it."""
    pool = random_pool(1, 8, 1, 64, 1)
    args = i32([[2, 3, 4]]), i32([2]), i32([1, 3]), 5
    k = [x.double() for x in mk.minisgl_load_kv_fp4(pool, 0, *args)][0][1:3]
    torch.use_deterministic_algorithms(True)
    try:
        got = mk.minisgl_load_kv_fp4(pool, 0, *args)
    finally:
        torch.use_deterministic_algorithms(False)
    for x in got:
        assert x.shape == (5, 1, 64) and torch.isnan(x).all(dim=(1, 2)).tolist() == [True, False, False, True, True]
    assert torch.equal(got[0][1:3].double(), k)


def test_exponents_of_a_pool():
    """numpy and torch integers as exponents, and what is none refused as any other argument."""
    pool = mk.KVPoolFP4.zeros(2, 4, 1, 64, k_exp=np.int64(-2), v_exp=torch.tensor([1, -3]))
    assert pool.k_exp == [-2, -2] and pool.v_exp == [1, -3]
    k = kv_like((4, 1, 64), 1).to(DEV)
    check_store(pool, 1, k, k, np.arange(4))
    with pytest.raises(mk.MinisglError, match="v_exp must be"):
        mk.KVPoolFP4.zeros(2, 4, 1, 64, v_exp=np.float32(1))


class Engine:
    """One layer of a serving engine over the 4-bit pool, by the public calls:
    slots, store, and extend or decode attention."""

    def __init__(self, B, W, pages, page, Hq, Hkv, d, seed):
        self.B, self.page, self.Hq, self.Hkv, self.d = B, page, Hq, Hkv, d
        self.dummy = pages * page
        self.pool = mk.KVPoolFP4.zeros(1, pages * page + 1, Hkv, d, page, k_exp=-2, v_exp=-2)
        self.table = torch.full((B, W), self.dummy, dtype=torch.int32, device=DEV)
        self.free = i32(np.random.default_rng(seed).permutation(pages))
        self.lens = i32([0] * B)
        self.sm = d ** -0.5

    def slots(self, extend, total):
        return mk.minisgl_build_slots(self.lens, extend, self.table, self.free, self.page, self.dummy, total)

    def finish(self, s):
        used = int(s.pages_used)
        assert used <= self.free.numel()
        self.free = self.free[used:].contiguous()
        self.lens = s.seq_lens.clone()

    def prefill(self, s, extend, q, k, v, total_kv):
        """Store the chunk, read all cached rows back as a small bf16 pool, attend."""
        mk.minisgl_store_kv_fp4(self.pool, 0, k, v, s.out_loc)
        rows = i32(range(total_kv))
        table = torch.zeros_like(self.table)
        packed = mk.minisgl_build_slots(torch.zeros_like(s.seq_lens), s.seq_lens, table, rows, 1, 0, total_kv)
        wide = torch.zeros((2, 1, total_kv, self.Hkv, self.d), dtype=torch.bfloat16, device=DEV)
        mk.minisgl_load_kv_fp4(self.pool, 0, self.table, s.seq_lens, packed.q_offsets, total_kv, wide[0, 0], wide[1, 0])
        return mk.minisgl_extend_attn(mk.KVPool(wide), 0, q, table, self.lens, extend, s.q_offsets, self.sm)


def test_prefill_in_chunks_then_decode_steps():
    """The operators as an engine runs them: two prefill chunks, then decode
    steps, against 64-bit attention over the definition's quantised values."""
    B, Hq, Hkv, d, page = 5, 16, 4, 128, 16
    eng = Engine(B, 288, 90, page, Hq, Hkv, d, 7)
    rng = np.random.default_rng(7)
    kept = [[] for _ in range(B)], [[] for _ in range(B)]  # the definition's K and V per request

    def new(extend, seed):
        T = int(sum(extend))
        q, k, v = (kv_like((T, h, d), seed + i).to(DEV) for i, h in enumerate((Hq, Hkv, Hkv)))
        at = 0
        for r, e in enumerate(extend):
            for x, keep in ((k, kept[0]), (v, kept[1])):
                c, sb = ref.quantise(ref.bf16_to_f64(x[at:at + e]), -2)
                keep[r].extend(ref.values(ref.pack(c), sb, -2))
            at += e
        return q, k, v

    for chunk in range(2):
        extend = rng.integers(0, 100, B)
        extend[chunk] = 0
        q, k, v = new(extend, 100 * chunk)
        T = int(extend.sum())
        s = eng.slots(i32(extend), T)
        total = sum(len(x) for x in kept[0])
        o = eng.prefill(s, i32(extend), q, k, v, total)
        # Extend attention rounds its weights to bf16 (half a step: 2^-8), and its output: values here
        # reach 8, where half a step is 2^-8 * 8 = 0.031, above the 0.02 that the library's tests use
        # for values around 0.5.  So the bound is counted per output, as for decode.
        got = o.double().cpu().numpy()
        for i, (r, p) in enumerate(zip(np.repeat(np.arange(B), extend), s.positions.tolist())):
            kk, vv = np.array(kept[0][r][:p + 1]), np.array(kept[1][r][:p + 1])
            want, mag, top = ref.decode(ref.bf16_to_f64(q[i:i + 1]), kk, vv, np.arange(p + 1)[None], [p + 1], eng.sm)
            bound = ref.decode_bound(want, mag, top, np.abs(vv).max(), p + 1, weight_step=2.0 ** -8)
            assert (np.abs(got[i:i + 1] - want) <= bound).all(), (chunk, i)
        eng.finish(s)
    for step in range(20):
        extend = [1] * B
        q, k, v = new(extend, 1000 + 10 * step)
        s = eng.slots(i32(extend), B)
        mk.minisgl_store_kv_fp4(eng.pool, 0, k, v, s.out_loc)
        o = mk.minisgl_decode_attn_fp4(eng.pool, 0, q, eng.table, s.seq_lens, eng.sm)
        lens = s.seq_lens.tolist()
        assert lens == [len(x) for x in kept[0]]
        n = max(lens)
        kk = np.zeros((B * n, Hkv, d))
        vv = np.zeros((B * n, Hkv, d))
        pt = np.zeros((B, n), dtype=int)
        for r in range(B):
            kk[r * n:r * n + lens[r]], vv[r * n:r * n + lens[r]] = kept[0][r], kept[1][r]
            pt[r, :lens[r]] = np.arange(r * n, r * n + lens[r])
        want, mag, top = ref.decode(ref.bf16_to_f64(q), kk, vv, pt, lens, eng.sm)
        bound = ref.decode_bound(want, mag, top, np.abs(vv).max(), n)
        assert (np.abs(o.double().cpu().numpy() - want) <= bound).all()
        eng.finish(s)
    live = {int(x) for r, n in enumerate(eng.lens.tolist()) for x in eng.table[r, :n].tolist()}
    assert len(live) == sum(eng.lens.tolist()) and eng.dummy not in live, "two tokens share a row"


def test_graph_of_a_decode_step_with_padding():
    """Slots, store and decode captured for a padded batch and replayed while
    the lengths advance in place; two graphs with workspaces of their own
    replayed at once on two streams."""
    B, Hq, Hkv, d = 6, 16, 8, 128
    steps = 4
    runs = []
    for _ in range(3):
        eng = Engine(B, 96, 60, 4, Hq, Hkv, d, 3)
        lens = i32([20, 0, 3, 40, -1, -1])
        pre = i32([20, 0, 3, 40, 0, 0])
        zero = torch.zeros(B, dtype=torch.int32, device=DEV)
        s = mk.minisgl_build_slots(zero, pre, eng.table, eng.free, 4, eng.dummy, 63)
        k0, v0 = kv_like((63, Hkv, d), 1).to(DEV), kv_like((63, Hkv, d), 2).to(DEV)
        mk.minisgl_store_kv_fp4(eng.pool, 0, k0, v0, s.out_loc)
        eng.free = eng.free[int(s.pages_used):].contiguous()
        one = torch.ones(B, dtype=torch.int32, device=DEV)
        q, k, v = (kv_like((B, h, d), 50 + h).to(DEV) for h in (Hq, Hkv, Hkv))
        q[5], k[5], v[5] = q[4], k[4], v[4]
        runs.append((eng, lens, one, q, k, v))

    def step(x):
        eng, lens, one, q, k, v = x
        s = mk.minisgl_build_slots(lens, one, eng.table, eng.free, 4, eng.dummy, B)
        mk.minisgl_store_kv_fp4(eng.pool, 0, k, v, s.out_loc)
        o = mk.minisgl_decode_attn_fp4(eng.pool, 0, q, eng.table, s.seq_lens, eng.sm)
        lens[:4] += 1
        eng.free.copy_(torch.roll(eng.free, -8))  # pages never handed out twice in these steps
        return o

    want = []
    for _ in range(steps):
        want.append(step(runs[0]).clone())
    graphs = []
    for x in runs[1:]:
        saved = [t.clone() for t in (x[1], x[0].free, x[0].table, x[0].pool.data, x[0].pool.scales)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(x)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = step(x)
        for t, y in zip((x[1], x[0].free, x[0].table, x[0].pool.data, x[0].pool.scales), saved):
            t.copy_(y)
        graphs.append((g, o, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(steps):
        for g, _, st in graphs:
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for _, o, _ in graphs:
            assert torch.equal(o, want[i]), f"step {i}"
