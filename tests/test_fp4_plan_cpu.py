"""The 4-bit decode's plan (csrc/decode_fp4_plan.h), compiled for the host:
which bytes of a token's scales its copies read, and which calls leave every
stream to one group of warps."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SHIM = """
#include "decode_fp4_plan.h"
using namespace minisgl::fp4;
extern "C" {
int block_heads_(int h) { return block_heads(h); }
int heads_of_block_(int h, int heads, int hb) { return heads_of_block(h, heads, hb); }
int scale_piece_(int heads, int sb) { return scale_piece(heads, sb); }
int piece_bytes_(int row, int off, int piece) { return piece_bytes(row, off, piece); }
int leave_whole_(int streams, int groups, int wide) { return leave_whole(streams, groups, wide); }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cc").write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "paged_kv_cache_row_gb300", "csrc"), str(d / "plan.cc"), "-o",
                    str(d / "plan.so")], check=True)
    return ctypes.CDLL(str(d / "plan.so"))


@pytest.mark.parametrize("d", [64, 128])
def test_scale_copies_read_each_byte_of_a_row_once_and_no_other(plan, d):
    """The copies of all head blocks, as the kernel issues them: a lane per
    piece of a full block, the block's heads given only by the plan."""
    sb = d // 16
    for H in list(range(1, 129)) + [4095, 4096]:
        heads = plan.block_heads_(H)
        assert heads == H if H <= 8 else 5 <= heads <= 8
        piece = plan.scale_piece_(heads, sb)
        assert piece in (sb, 16) and heads * sb % piece == 0
        read = []
        for hb in range(-(-H // heads)):
            nh = plan.heads_of_block_(H, heads, hb)
            assert 1 <= nh <= heads and (hb > 0 or nh == heads)
            for off in range(0, heads * sb, piece):
                n = plan.piece_bytes_(nh * sb, off, piece)
                assert n % sb == 0  # a copy of d/16 bytes at a time ends with it
                read += range(hb * heads * sb + off, hb * heads * sb + off + n)
        assert read == list(range(H * sb)), H
        assert plan.piece_bytes_(heads * sb, 1 << 30, piece) == 0  # lanes without a piece


@pytest.mark.parametrize("groups", [132, 152, 304, 608, 2432])
def test_streams_are_left_whole_in_narrow_tables_only(plan, groups):
    """A group that has a stream for itself takes up to the table's width alone,
    while every other may be done after one tile: only a few tiles may depend
    on how the lengths happen to lie, however close the batch is to the number
    of groups."""
    for streams in sorted({1, groups // 3, groups // 2, groups - 3, groups - 1, groups, groups + 1, 2 * groups}):
        for wide in list(range(40)) + [256, 1024, 1 << 25]:
            whole = plan.leave_whole_(streams, groups, wide)
            assert not whole or (streams <= groups and wide <= 8), (streams, wide)
            if wide <= 5:
                assert whole == (streams <= groups)
