"""The 8-bit pool and the rotary tables without a GPU: the tests' own 64-bit
definitions against torch's formats and closed forms, the frequencies (computed
on the host), and the calls' refusals (checked on the host before any device
work; the pointers are never dereferenced)."""
import ctypes
import math
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

import paged_kv_cache_row_gb300 as mk
from tests import fp8_ref as ref

FAKE = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_row_gb300 import build
    build.build()
    return mk.load_library()


# --------------------------------------------------------------------------- #
# the definitions
# --------------------------------------------------------------------------- #
def test_elements_are_torchs():
    """Nearest, ties to even, on every bf16 up to 448 in size."""
    x = torch.arange(0, 0x7F80, dtype=torch.int16).view(torch.bfloat16)
    x = torch.cat([x, -x])
    x = x[x.float().abs() <= 448]
    assert np.array_equal(ref.element(x.double().numpy()), x.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert ref.element(np.array([449.0, -1e9, np.nan, np.inf])).tolist() == [0x7E, 0xFE, 0x7F, 0x7F]


def test_needed_exponent():
    for e in (-120, -3, 0, 7, 119):
        top = 448 * 2.0 ** e
        assert ref.needed(np.array([top, np.nextafter(top, 0), np.nextafter(top, np.inf), top / 2])).tolist() == \
            [e, e, min(e + 1, 119), max(e - 1, -120)]
    assert ref.needed(np.array([0.0, 1e-45, 3.4e38])).tolist() == [-120, -120, 119]


def test_a_block_that_grows():
    """Block of 4 rows: 1.0 needs 2^-8; 448 then needs 2^0, and 1.0 is kept exactly, 2^-9 is kept as a subnormal."""
    codes, exps = np.zeros((8, 1, 2), np.uint8), np.zeros((2, 1), int)
    ref.store(codes, exps, [4, 5], np.array([[[1.0, 2.0 ** -9]], [[0.5, 2.0 ** -11]]]), 4)
    assert exps[1, 0] == -8
    ref.store(codes, exps, [6], np.array([[[448.0, -3.0]]]), 4)
    assert exps[1, 0] == 0 and exps[0, 0] == 0
    assert ref.values(codes, exps, 4)[4:7, 0].tolist() == [[1.0, 2.0 ** -9], [0.5, 0.0], [448.0, -3.0]]
    ref.store(codes, exps, [4], np.array([[[0.25, 0.125]]]), 4)  # the block begins anew
    assert exps[1, 0] == -10


def test_values_are_bf16():
    v = ref.values(np.tile(np.arange(256, dtype=np.uint8), (240, 1, 1)), np.arange(-120, 120)[:, None], 1)
    got = torch.from_numpy(v).to(torch.bfloat16).double().numpy()
    assert np.array_equal(got, v, equal_nan=True)


def test_error_of_a_block():
    """Half a step of e4m3 (2^-4) of a value, and half a subnormal step of its
    block: 2^-10 * 2^e, with 2^e < max / 224."""
    x = np.random.default_rng(0).normal(size=(64, 3, 64)) * np.exp(np.random.default_rng(1).normal(size=(3, 64)))
    codes, exps = np.zeros((64, 3, 64), np.uint8), np.zeros((4, 3), int)
    ref.store(codes, exps, np.arange(64), x, 16)
    top = np.repeat(np.abs(x).reshape(4, 16, 3, 64).max((1, 3)), 16, 0)[..., None]
    assert (np.abs(ref.values(codes, exps, 16) - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * top / 224)).all()


# --------------------------------------------------------------------------- #
# frequencies
# --------------------------------------------------------------------------- #
KINDS = [dict(), dict(kind="linear", factor=8.0), dict(kind="ntk", factor=4.0),
         dict(kind="bands", factor=8.0, original_positions=8192), dict(kind="yarn", factor=32.0, original_positions=4096),
         dict(kind="yarn", factor=40.0, original_positions=4096, attention_factor=1.0),
         dict(kind="yarn", factor=2.0, original_positions=2, slow_turns=0.5, fast_turns=0.6),
         dict(kind="bands", factor=3.0, original_positions=100, slow_turns=2.0, fast_turns=30.0)]


@pytest.mark.parametrize("base", [10000.0, 500000.0])
@pytest.mark.parametrize("rotary", [16, 48, 128, 256])
@pytest.mark.parametrize("kind", KINDS, ids=[str(i) + k.get("kind", "plain") for i, k in enumerate(KINDS)])
def test_frequencies(lib, kind, rotary, base):
    """turns / 2^64 * 2 pi is theta: within 2^-64 turns for the rounding, and
    2^-44 of it for a dozen operations in double on either side (a power's error
    is its logarithm's, below 32, times 2^-53: 2^-48)."""
    rope = mk.Rope(rotary, base, **kind)
    theta, attention = ref.frequencies(rotary, base, kind.get("kind", "plain"), kind.get("factor", 1.0),
                                       kind.get("original_positions", 0), kind.get("slow_turns", 1.0),
                                       kind.get("fast_turns"), kind.get("attention_factor"))
    got = np.array([t / 2.0 ** 64 * 2 * math.pi for t in rope.turns])
    assert np.abs(got - theta).max() <= 2.0 ** -60 + 2.0 ** -44
    assert (np.abs(got - theta) <= 2.0 ** -60 + 2.0 ** -44 * np.array(theta)).all()
    assert abs(rope.attention_factor - attention) <= 2.0 ** -23 * attention


PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def exact_frequencies(n, base, kind, factor, origin, slow, fast):
    """The definition with 60 digits."""
    with localcontext() as c:
        c.prec = 60
        base, f, origin, slow, fast = (Decimal(x) for x in (base, factor, origin, slow, fast))
        if kind == "ntk":
            base *= (f.ln() * n / (n - 2)).exp()
        ln = base.ln()
        if kind == "yarn":
            at = [n * (origin / (2 * PI * t)).ln() / (2 * ln) for t in (fast, slow)]
            lo, hi = max(0, math.floor(at[0])), min(n - 1, math.ceil(at[1]))
            hi = hi if hi > lo else lo + Decimal("0.001")
        out = []
        for j in range(n // 2):
            theta, s = (-2 * j * ln / n).exp(), Decimal(kind == "linear")
            if kind == "bands":
                s = 1 - min(Decimal(1), max(Decimal(0), (origin * theta / (2 * PI) - slow) / (fast - slow)))
            if kind == "yarn":
                s = min(Decimal(1), max(Decimal(0), Decimal(j - lo) / Decimal(hi - lo)))
            out.append(s * theta / f + (1 - s) * theta)
        return out


@pytest.mark.parametrize("base", [1.5, 100.0, 10000.0, 500000.0, 1e6, 1e30])
@pytest.mark.parametrize("kind,factor,origin,slow,fast", [
    ("plain", 1.0, 0, 1, 32), ("linear", 3.7, 0, 1, 32), ("ntk", 8.0, 0, 1, 32), ("ntk", 1e6, 0, 1, 32),
    ("bands", 8.0, 8192, 1, 4), ("bands", 7.7, 3.0, 1, 4), ("bands", 3.0, 100, 2.0, 2.001), ("yarn", 32.0, 4096, 1, 32),
    ("yarn", 2.3, 2, 0.5, 0.6), ("yarn", 40.0, 100000, 1, 32)])
def test_frequencies_are_as_near_as_the_header_says(lib, base, kind, factor, origin, slow, fast):
    """Within 2^-50 radians a position, and for bands 2^-49 fast / (fast - slow)."""
    bound = 2.0 ** -49 * fast / (fast - slow) if kind == "bands" else 2.0 ** -50
    for n in (16, 48, 96, 128, 256):
        turns = mk.Rope(n, base, kind, factor=factor, original_positions=origin, slow_turns=slow, fast_turns=fast).turns
        want = exact_frequencies(n, base, kind, factor, origin, slow, fast)
        with localcontext() as c:
            c.prec = 60
            off = [abs(Decimal(t) * 2 * PI / 2 ** 64 - w) for t, w in zip(turns, want)]
        assert max(off) <= Decimal(bound), (n, off.index(max(off)), float(max(off)) * 2.0 ** 53)


def test_frequency_scalings():
    """What each kind is for: the fastest pair and the slowest one."""
    plain = mk.Rope(128).turns
    lin, ntk = mk.Rope(128, kind="linear", factor=8.0).turns, mk.Rope(128, kind="ntk", factor=8.0).turns
    bands, yarn = (mk.Rope(128, kind=k, factor=8.0, original_positions=4096).turns for k in ("bands", "yarn"))
    for t, first in ((lin, 8), (ntk, 1), (bands, 1), (yarn, 1)):
        assert abs(plain[0] / t[0] - first) < 1e-9 and abs(plain[-1] / t[-1] - 8) < 1e-9


BAD_ROPES = [dict(rotary_dim=8), dict(rotary_dim=272), dict(rotary_dim=100), dict(rotary_dim=-16), dict(base=1.0),
             dict(base=math.nan), dict(base=math.inf), dict(kind="linear", factor=0.5),
             dict(kind="ntk", factor=math.nan), dict(kind="spiral"), dict(kind="yarn", factor=2.0),
             dict(kind="bands", factor=2.0, original_positions=math.inf),
             dict(kind="bands", factor=2.0, original_positions=4096, slow_turns=4.0),
             dict(kind="yarn", factor=2.0, original_positions=4096, slow_turns=0.0), dict(attention_factor=0.0),
             dict(attention_factor=-1.0), dict(attention_factor=math.nan), dict(attention_factor=1e9)]


@pytest.mark.parametrize("bad", BAD_ROPES, ids=str)
def test_bad_ropes_are_refused(lib, bad):
    with pytest.raises(mk.MinisglError):
        mk.Rope(**{**dict(rotary_dim=64), **bad})


def test_rope_table_refusals(lib):
    turns = (ctypes.c_uint64 * 128)()
    f = lib.minisgl_rope_table
    assert f(None, 1.0, 64, FAKE, 4, 2 * FAKE, None) == -1
    for dim in (0, 8, 40, 272):
        assert f(turns, 1.0, dim, FAKE, 4, 2 * FAKE, None) == -4
    assert f(turns, 1.0, 64, FAKE, -1, 2 * FAKE, None) == -1
    assert f(turns, 1.0, 64, None, 4, 2 * FAKE, None) == -1 and f(turns, 1.0, 64, FAKE, 4, None, None) == -1
    assert f(turns, 1.0, 64, FAKE, 4, 2 * FAKE + 8, None) == -3
    assert f(turns, 1.0, 64, FAKE + 16, 4, FAKE, None) == -1  # out overlaps positions
    assert f(turns, 1.0, 64, FAKE, 0, FAKE, None) == 0
    assert b"rope_table" in (lib.minisgl_rope_table(None, 1.0, 64, FAKE, 4, FAKE, None), lib.minisgl_last_error())[1]
    g = lib.minisgl_rope_frequencies
    att = ctypes.c_float()
    assert g(None, turns, ctypes.byref(att)) == -1
    desc = mk._RopeDesc(kind=0, rotary_dim=64, base=1e4)
    assert g(ctypes.byref(desc), None, ctypes.byref(att)) == -1 and g(ctypes.byref(desc), turns, None) == -1
    assert g(ctypes.byref(mk._RopeDesc(kind=7, rotary_dim=64, base=1e4)), turns, ctypes.byref(att)) == -1


# --------------------------------------------------------------------------- #
# refusals of the pool's calls
# --------------------------------------------------------------------------- #
def _desc(**kw):
    d = dict(k_data=FAKE, v_data=FAKE, k_scale=FAKE, v_scale=FAKE, data_layer_stride=100 * 1024,
             data_row_stride=1024, scale_layer_stride=100 * 8, scale_block_stride=8, num_layers=1, num_rows=100,
             num_kv_heads=8, head_dim=128, page_size=16, block_tokens=16, dtype=mk.MINISGL_FP8)
    d.update(kw)
    return mk._PoolFP8Desc(**d)


BAD_POOLS = [(dict(dtype=2), -2), (dict(k_data=0), -1), (dict(v_data=0), -1), (dict(k_scale=0), -1),
             (dict(v_scale=0), -1), (dict(head_dim=96), -4), (dict(num_kv_heads=0), -3), (dict(num_rows=0), -3),
             (dict(num_layers=0), -3),
             (dict(num_kv_heads=4097, data_row_stride=1 << 20, scale_block_stride=1 << 20), -4),
             (dict(block_tokens=8), -4), (dict(block_tokens=0), -4), (dict(block_tokens=128, page_size=128), -4),
             (dict(page_size=0), -3), (dict(page_size=24), -3), (dict(block_tokens=64), -3),
             (dict(data_row_stride=1008), -3), (dict(data_row_stride=1032), -3), (dict(scale_block_stride=4), -3),
             (dict(scale_block_stride=10), -3), (dict(num_kv_heads=5, scale_block_stride=4), -3),
             (dict(data_row_stride=1 << 31), -4), (dict(scale_block_stride=1 << 31), -4),
             (dict(k_data=FAKE + 8), -3), (dict(data_layer_stride=8), -3), (dict(k_scale=FAKE + 2), -3),
             (dict(v_scale=FAKE + 1), -3), (dict(scale_layer_stride=6), -3)]


@pytest.mark.parametrize("change,code", BAD_POOLS, ids=[str(b[0]) for b in BAD_POOLS])
def test_bad_pools_are_refused_by_every_call(lib, change, code):
    d = ctypes.byref(_desc(**change))
    assert lib.minisgl_store_kv_fp8(d, 0, FAKE, FAKE, 1024, 1024, FAKE, 4, None) == code
    assert lib.minisgl_rope_store_kv_fp8(d, 0, FAKE, 16, 2048, FAKE, 2048, FAKE, FAKE, 1024, 1024, FAKE, FAKE, 99, 64,
                                         0, FAKE, 4, None) == code
    assert lib.minisgl_load_kv_fp8(d, 0, FAKE, 4, 32, 32, FAKE, FAKE, 9, FAKE, FAKE, 1024, 1024, None) == code
    assert lib.minisgl_decode_attn_fp8(d, 0, FAKE, 16, FAKE, 4, 32, 32, FAKE, 0.1, FAKE, FAKE, 1 << 20, 0,
                                       None) == code
    assert lib.minisgl_last_error()


def _varied(f, good):
    return lambda i, x: f(*(good[:i] + [x] + good[i + 1:]))


def test_store_refusals(lib):
    call = _varied(lib.minisgl_store_kv_fp8, [ctypes.byref(_desc()), 0, FAKE, FAKE, 1024, 1024, FAKE, 4, None])
    assert call(0, None) == -1 and call(1, 1) == -1 and call(1, -1) == -1 and call(7, -1) == -1
    for i in (2, 3, 6):
        assert call(i, None) == -1
    assert call(2, FAKE + 8) == -3 and call(3, FAKE + 2) == -3 and call(4, 1016) == -3 and call(5, 1028) == -3
    assert call(7, 1 << 24) == -4
    assert call(7, 0) == 0


def test_rope_store_refusals(lib):
    good = [ctypes.byref(_desc()), 0, FAKE, 16, 2048, 2 * FAKE, 2048, FAKE, FAKE, 1024, 1024, FAKE, FAKE, 99, 64, 0,
            FAKE, 4, None]
    call = _varied(lib.minisgl_rope_store_kv_fp8, good)
    assert call(0, None) == -1 and call(1, 1) == -1 and call(17, -1) == -1
    for i in (2, 5, 7, 8, 11, 12, 16):
        assert call(i, None) == -1
    assert call(3, -1) == -1 and call(13, 0) == -1
    for dim in (0, 8, 24, 144, 256):
        assert call(14, dim) == -4
    assert call(2, FAKE + 8) == -3 and call(5, FAKE + 8) == -3 and call(7, FAKE + 8) == -3 and call(12, FAKE + 4) == -3
    assert call(4, 2040) == -3 and call(6, 2052) == -3 and call(9, 1016) == -3 and call(10, 1028) == -3
    assert call(3, 1 << 30) == -3  # rows of q wider than its stride
    wide = list(good)
    wide[3], wide[4], wide[6], wide[17] = 1 << 17, 1 << 24, 1 << 24, 1 << 11  # 2^24 channels of q in each of 2^11 tokens
    assert lib.minisgl_rope_store_kv_fp8(*wide) == -4
    # q_out may be q itself, and nothing else of it
    assert call(5, FAKE + 256) == -1 and call(5, FAKE - 256) == -1 and call(5, FAKE + 3 * 4096) == -1
    shifted = list(good)
    shifted[5], shifted[6] = FAKE, 4096
    assert lib.minisgl_rope_store_kv_fp8(*shifted) == -1
    assert call(17, 0) == 0
    assert b"rope_store_kv_fp8" in (call(3, -1), lib.minisgl_last_error())[1]


def test_rope_store_refuses_queries_over_k_or_v(lib):
    """q_out, q itself or not, on a row of k or of v: the first, the last, and by 16 bytes between two others."""
    good = [ctypes.byref(_desc()), 0, FAKE, 16, 8192, 2 * FAKE, 8192, 3 * FAKE, 4 * FAKE, 8192, 8192, FAKE, FAKE, 99, 64, 0,
            FAKE, 4, None]  # 4 KB of q and 2 KB of k and v, in rows of 16 KB
    for i in (7, 8):
        for out in (2 * FAKE, FAKE):
            for off in (0, 4096 - 16, 16 - 2048, 3 * 16384 + 4000, -3 * 16384, 16384 + 16):
                bad = list(good)
                bad[5], bad[i] = out, out + off
                assert lib.minisgl_rope_store_kv_fp8(*bad) == -1, (i, off)
                assert b"q_out overlaps k or v" in lib.minisgl_last_error()


def test_load_refusals(lib):
    call = _varied(lib.minisgl_load_kv_fp8, [ctypes.byref(_desc()), 0, FAKE, 4, 32, 32, FAKE, FAKE, 9, FAKE, FAKE, 1024,
                                             1024, None])
    assert call(1, 1) == -1 and call(3, -1) == -1 and call(3, 4097) == -1 and call(8, -1) == -1
    for i in (0, 2, 6, 7, 9, 10):
        assert call(i, None) == -1
    assert call(4, 31) == -3 and call(5, -1) == -3
    assert call(9, FAKE + 8) == -3 and call(10, FAKE + 4) == -3 and call(11, 1016) == -3 and call(12, 1028) == -3
    assert call(3, 0) == 0 and call(8, 0) == 0


def test_decode_refusals(lib):
    need = lib.minisgl_decode_workspace_bytes(4, 16, 8, 128, 2)
    good = [ctypes.byref(_desc()), 0, FAKE, 16, FAKE, 4, 32, 32, FAKE, 0.1, FAKE, FAKE, need, 0, None]
    call = _varied(lib.minisgl_decode_attn_fp8, good)
    assert call(0, None) == -1 and call(1, 1) == -1
    assert call(3, 12) == -3 and call(3, 0) == -3 and call(3, 8 * 17) == -4 and call(5, -1) == -1 and call(5, 4097) == -1
    for i in (2, 4, 8, 10):
        assert call(i, None) == -1
    assert call(2, FAKE + 8) == -3 and call(10, FAKE + 2) == -3 and call(6, 31) == -3 and call(7, -1) == -3
    assert call(11, None) == -6 and call(11, FAKE + 128) == -6 and call(12, need - 1) == -6
    assert b"decode_attn_fp8" in lib.minisgl_last_error()
    assert call(13, -1) == -1
    wide = list(good)
    for width in ((1 << 30) + 1, (1 << 31) - 1):
        wide[6] = wide[7] = width
        assert lib.minisgl_decode_attn_fp8(*wide) == -4
    assert call(5, 0) == 0


def test_pool_bytes():
    assert mk.kv_pool_fp8_bytes(32, 8, 128, 1000, 16) == 2 * 32 * (8 * 128 * 1000 + 8 * 63)
    assert mk.kv_pool_fp8_bytes(1, 5, 64, 10, 1) == 2 * (5 * 64 * 10 + 8 * 10)


def test_pools_on_the_cpu_are_refused():
    with pytest.raises(mk.MinisglError):
        mk.KVPoolFP8(torch.zeros(2, 1, 32, 8, 64, dtype=torch.uint8), torch.zeros(2, 1, 2, 8, dtype=torch.uint8), 16, 16)
