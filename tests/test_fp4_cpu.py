"""The 4-bit pool without a GPU: the tests' own 64-bit definitions against
torch's formats and closed forms, and the calls' refusals (checked on the host
before any device work; the pointers are never dereferenced)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import paged_kv_cache_row_gb300 as mk
from tests import fp4_ref as ref

FAKE = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_row_gb300 import build
    build.build()
    return mk.load_library()


def test_e4m3_table_is_torchs():
    got = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, ref.E4M3)


def test_scale_rounding_is_torchs():
    """Nearest, ties to even, on every positive bf16 up to 448 (times 1, exact)."""
    x = torch.arange(1, 0x7F80, dtype=torch.int16).view(torch.bfloat16)
    x = x[x.float() <= 448]
    want = x.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.nearest_even(x.double().numpy(), ref.E4M3), want)


def test_quantise_borders():
    """Elements on every border of e2m1 under scale 1 (the block's largest is 6)."""
    x = np.array([6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -5, -3.5, -2.5, -1.75, -1.25, -0.75, -0.25, -0.0])
    codes, sb = ref.quantise(x, 0)
    assert ref.E4M3[sb[0]] == 1
    got = ref.values(ref.pack(codes), sb, 0)
    assert got.tolist() == [6, 4, 4, 2, 2, 1, 1, 0, -4, -4, -2, -2, -1, -1, 0, 0]
    assert codes[-1] == 8 and codes[-2] == 8


def test_quantised_values_are_bf16():
    data = np.arange(256, dtype=np.uint8)[None].repeat(127, 0).reshape(127, 32, 8)
    scales = np.arange(127, dtype=np.uint8)[:, None].repeat(32, 1)[..., None]
    v = ref.values(data, scales, 3)
    assert np.array_equal(torch.from_numpy(v).to(torch.bfloat16).double().numpy(), v)


def test_quantisation_error_bound():
    """|value - x| is at most a quarter of the block's largest: one e2m1 step is
    at most 2 of 6, the scale is at most 1/16 off (2^-6 and above)."""
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.normal(size=(500, 128))).to(torch.bfloat16).double().numpy()
    codes, sb = ref.quantise(x, -4)
    err = np.abs(ref.values(ref.pack(codes), sb, -4) - x).reshape(500, -1, 16).max(-1)
    assert (err <= 0.25 * np.abs(x).reshape(500, -1, 16).max(-1)).all()


def test_slots_reference_example():
    """Two requests and a padding request, pages of 4: request 0 has 3 cached
    tokens in page 7 and fills it before it takes a new page."""
    table = np.full((3, 8), -5)
    table[0, :3] = [28, 29, 30]
    t, loc, pos, off, ends, used = ref.build_slots([3, 0, -1], [3, 5, 1], table, [2, 9, 4, 6], 4, 99, 11)
    assert t.tolist() == [[28, 29, 30, 31, 8, 9, -5, -5], [36, 37, 38, 39, 16, -5, -5, -5], [99] + [-5] * 7]
    assert loc.tolist() == [31, 8, 9, 36, 37, 38, 39, 16, 99, 99, 99]
    assert pos.tolist() == [3, 4, 5, 0, 1, 2, 3, 4, 0, 0, 0]
    assert off.tolist() == [0, 3, 8, 9] and ends.tolist() == [6, 5, 1] and used == 3


def _desc(**kw):
    d = dict(k_data=FAKE, v_data=FAKE, k_scale=FAKE, v_scale=FAKE, data_layer_stride=100 * 512,
             data_row_stride=512, scale_layer_stride=100 * 64, scale_row_stride=64, num_layers=1, num_rows=100,
             num_kv_heads=8, head_dim=128, page_size=1, dtype=mk.MINISGL_FP4, k_exp=0, v_exp=0)
    d.update(kw)
    return mk._PoolFP4Desc(**d)


BAD_POOLS = [(dict(dtype=1), -2), (dict(k_data=0), -1), (dict(v_scale=0), -1), (dict(head_dim=96), -4),
             (dict(num_kv_heads=0), -3), (dict(num_rows=0), -3), (dict(num_layers=0), -3),
             (dict(num_kv_heads=4097, data_row_stride=1 << 20, scale_row_stride=1 << 20), -4),
             (dict(data_row_stride=496), -3), (dict(data_row_stride=520), -3), (dict(scale_row_stride=56), -3),
             (dict(scale_row_stride=68), -3), (dict(k_data=FAKE + 8), -3), (dict(data_layer_stride=8), -3),
             (dict(k_scale=FAKE + 4), -3), (dict(scale_layer_stride=4), -3), (dict(k_exp=65), -1),
             (dict(v_exp=-65), -1)]


@pytest.mark.parametrize("change,code", BAD_POOLS, ids=[str(b[0]) for b in BAD_POOLS])
def test_bad_pools_are_refused_by_every_call(lib, change, code):
    d = ctypes.byref(_desc(**change))
    assert lib.minisgl_store_kv_fp4(d, 0, FAKE, FAKE, 1024, 1024, FAKE, 4, None) == code
    assert lib.minisgl_load_kv_fp4(d, 0, FAKE, 4, 32, 32, FAKE, FAKE, 9, FAKE, FAKE, 1024, 1024, None) == code
    assert lib.minisgl_decode_attn_fp4(d, 0, FAKE, 16, FAKE, 4, 32, 32, FAKE, 0.1, FAKE, FAKE, 1 << 20, 0,
                                       None) == code
    assert lib.minisgl_last_error()


def test_store_refusals(lib):
    d = ctypes.byref(_desc())
    f = lib.minisgl_store_kv_fp4
    assert f(None, 0, FAKE, FAKE, 1024, 1024, FAKE, 4, None) == -1
    assert f(d, 1, FAKE, FAKE, 1024, 1024, FAKE, 4, None) == -1
    assert f(d, 0, FAKE, FAKE, 1024, 1024, FAKE, -1, None) == -1
    assert f(d, 0, None, FAKE, 1024, 1024, FAKE, 4, None) == -1
    assert f(d, 0, FAKE, FAKE, 1024, 1024, None, 4, None) == -1
    assert f(d, 0, FAKE + 8, FAKE, 1024, 1024, FAKE, 4, None) == -3
    assert f(d, 0, FAKE, FAKE, 1016, 1024, FAKE, 4, None) == -3
    assert f(d, 0, FAKE, FAKE, 1024, 1028, FAKE, 4, None) == -3
    assert f(d, 0, FAKE, FAKE, 1024, 1024, FAKE, 1 << 24, None) == -4
    assert f(d, 0, FAKE, FAKE, 1024, 1024, FAKE, 0, None) == 0


def test_load_refusals(lib):
    d = ctypes.byref(_desc())
    f = lib.minisgl_load_kv_fp4
    good = [d, 0, FAKE, 4, 32, 32, FAKE, FAKE, 9, FAKE, FAKE, 1024, 1024, None]

    def call(i, x):
        return f(*(good[:i] + [x] + good[i + 1:]))
    assert call(3, -1) == -1 and call(3, 4097) == -1 and call(8, -1) == -1
    for i in (2, 6, 7, 9, 10):
        assert call(i, None) == -1
    assert call(4, 31) == -3 and call(5, -1) == -3
    assert call(9, FAKE + 8) == -3 and call(11, 1016) == -3 and call(12, 1028) == -3
    assert call(3, 0) == 0 and call(8, 0) == 0


def test_decode_refusals(lib):
    d = ctypes.byref(_desc())
    f = lib.minisgl_decode_attn_fp4
    need = lib.minisgl_decode_workspace_bytes(4, 16, 8, 128, 2)
    good = [d, 0, FAKE, 16, FAKE, 4, 32, 32, FAKE, 0.1, FAKE, FAKE, need, 0, None]

    def call(i, x):
        return f(*(good[:i] + [x] + good[i + 1:]))
    assert call(3, 12) == -3 and call(3, 8 * 17) == -4 and call(5, -1) == -1 and call(5, 4097) == -1
    for i in (2, 4, 8, 10):
        assert call(i, None) == -1
    assert call(2, FAKE + 8) == -3 and call(10, FAKE + 2) == -3 and call(6, 31) == -3
    assert call(11, None) == -6 and call(11, FAKE + 128) == -6 and call(12, need - 1) == -6
    assert b"decode_attn_fp4" in lib.minisgl_last_error()
    assert call(13, -1) == -1
    wide = list(good)
    for width in ((1 << 30) + 1, (1 << 31) - 1):
        wide[6], wide[7] = 1 << 31, width
        assert f(*wide) == -4
    assert call(5, 0) == 0


def test_slots_refusals(lib):
    f = lib.minisgl_build_slots
    at = [FAKE + (i << 24) for i in range(9)]  # apart from one another
    good = [at[0], at[1], 4, at[2], 32, 32, at[3], 10, 16, 99, at[4], at[5], at[6], at[7], at[8], 20, None]

    def call(*pairs):
        args = list(good)
        for i, x in pairs:
            args[i] = x
        return f(*args)
    assert call((2, -1)) == -1 and call((2, 4097)) == -1 and call((15, -1)) == -1 and call((7, -1)) == -1
    assert call((15, (1 << 30) + 1)) == -1
    assert call((8, 0)) == -1 and call((8, (1 << 20) + 1)) == -1 and call((9, -1)) == -1
    for i in (0, 1, 3, 6, 10, 11, 12, 13, 14):
        assert call((i, None)) == -1
    assert call((4, 31)) == -3 and call((5, -1)) == -3 and call((5, (1 << 30) + 1), (4, 1 << 31)) == -3
    # outputs on inputs, and on one another
    assert call((13, at[0])) == -1 and b"overlaps an input" in lib.minisgl_last_error()
    assert call((13, at[0] + 12)) == -1 and call((10, at[3] + 36)) == -1 and call((3, at[1] - 500)) == -1
    assert call((11, at[4] + 76)) == -1 and b"two outputs" in lib.minisgl_last_error()


def test_binding_refuses_host_tensors(lib):
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(mk.MinisglError, match="CUDA"):
        mk.minisgl_build_slots(i, i, i.reshape(4, 1), i, 1, 0, 4)
    with pytest.raises(mk.MinisglError, match="shape"):
        mk.KVPoolFP4(torch.zeros(2, 4, dtype=torch.uint8), torch.zeros(2, 4, dtype=torch.uint8))
    with pytest.raises(mk.MinisglError, match="CUDA"):
        mk.KVPoolFP4.zeros(1, 8, 2, 64, device="cpu")


def test_pool_bytes():
    assert mk.kv_pool_fp4_bytes(32, 8, 128, 1000) == 2 * 32 * 8 * 72 * 1000
    assert mk.kv_pool_bytes(32, 8, 128, 1000) / mk.kv_pool_fp4_bytes(32, 8, 128, 1000) == 256 / 72


def _code(name):
    """A CUDA source without its comments."""
    path = os.path.join(os.path.dirname(os.path.abspath(mk.__file__)), "csrc", name)
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)


SOURCES = ["build_slots.cu", "store_kv_fp4.cu", "fp4.cuh", "decode_fp4.cu", "decode_fp4.cuh", "decode_fp4_kernel.cuh"]


@pytest.mark.parametrize("name", SOURCES)
def test_early_started_kernels_load_coherently(name):
    """These kernels are resident while the one before them may still write
    what they read (lengths, slots, new rows, the pool): a non-coherent load
    wants memory that does not change for the kernel's whole life."""
    assert not re.findall(r"__ldg|ld_nc\w*|\.global\.nc", _code(name))


def test_slots_start_no_kernel_early():
    """The older kernels read page_table, out_loc and lengths with non-coherent
    loads, so they must not be resident while build_slots writes them."""
    code = _code("build_slots.cu")
    assert "pdl_wait()" in code and "pdl_launch_dependents" not in code


@pytest.mark.parametrize("e", [3, np.int64(3), np.int8(3), torch.tensor(3), [3, 3], (3, 3), np.array([3, 3]),
                               torch.tensor([3, 3]), [np.int32(3), torch.tensor(3)]], ids=repr)
def test_exponents_of_any_integer_kind(e):
    assert mk._exponents(e, 2, "k_exp") == [3, 3]


@pytest.mark.parametrize("e", [None, 1.5, [0.5, 0], np.float32(1), "12", [1], [1, 2, 3], 65, [0, -65], [0, None],
                               [0, float("nan")], [0, float("inf")], torch.tensor(0.5)], ids=repr)
def test_exponents_refused(e):
    with pytest.raises(mk.MinisglError, match="k_exp must be"):
        mk._exponents(e, 2, "k_exp")


def test_load_starts_no_kernel_early():
    """minisgl_store_kv may put the loaded rows into a bf16 pool, and reads new
    rows with non-coherent loads."""
    store, load = _code("store_kv_fp4.cu").split("load_kv_fp4_kernel(", 1)
    assert "pdl_launch_dependents()" in store
    assert "pdl_wait()" in load and "pdl_launch_dependents" not in load
