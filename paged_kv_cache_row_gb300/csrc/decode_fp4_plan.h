// decode_fp4_plan.h -- how decode_fp4_kernel cuts the KV heads of a row into
// blocks, which bytes of a token's scales each copy takes, and which calls
// leave every stream whole.
//
// Plain C++ without CUDA, so that the tests compile these functions for the
// host and check every head count.
#pragma once

namespace minisgl {
namespace fp4 {

// Heads of a block: ceil(H / 8) blocks of one size.  The last has the heads
// that are left, from one to all of them (25 heads: 7, 7, 7, 4; 57: seven
// blocks of 8 and one head).
constexpr int block_heads(int num_kv_heads) {
    const int blocks = (num_kv_heads + 7) / 8;
    return (num_kv_heads + blocks - 1) / blocks;
}
constexpr int heads_of_block(int num_kv_heads, int heads, int hb) {
    return num_kv_heads - hb * heads < heads ? num_kv_heads - hb * heads : heads;
}

// A token's scales of a full block (`heads` heads of sb bytes) are copied in
// pieces of this size.
constexpr int scale_piece(int heads, int sb) { return heads * sb % 16 == 0 ? 16 : sb; }

// How much of the piece that starts at `off` lies in a block whose scales are
// `row` bytes: all of it, none, or in a short last block a part (11 heads at
// head_dim 128 are blocks of 48 and 40 bytes, so the third piece has 8).  What
// follows is the next row, or the end of the caller's memory.
constexpr int piece_bytes(int row, int off, int piece) {
    return off >= row ? 0 : row - off < piece ? row - off : piece;
}

// Whether every stream (request and block of heads) is left to one group of
// warps: no schedule to sum, no partials, no merge launch, which saves about the
// time of 5 tiles.  A group then has up to `wide` tiles (the page table's width)
// one after the other instead of its share of all tiles.  The lengths are on
// the device, so the rule has to hold for the worst of them: a few requests as
// long as the table is wide among short ones.  Hence few tiles, and not many
// more groups than streams.  Whole / split in a graph, 8 KV heads, d 128, 256
// requests on 304 groups, in tables of 5, 8, 16 and 32 tiles (us):
//   all as long as the table       13.1/17.9  18.7/23.9  35.0/38.9  63.4/63.2
//   evenly spread up to it         11.3/16.9  15.8/19.8  27.3/31.6  51.4/48.9
//   one of them, the others 1 tile  9.7/10.2  13.2/10.4  22.6/11.3  41.3/12.5
constexpr int WHOLE_TILES = 8;
constexpr bool leave_whole(long long streams, long long groups, long long wide) {
    return streams <= groups && wide <= WHOLE_TILES && (wide - 5) * groups <= wide * streams;
}

}  // namespace fp4
}  // namespace minisgl
