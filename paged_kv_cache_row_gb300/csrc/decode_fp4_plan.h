// decode_fp4_plan.h -- how decode_fp4_kernel cuts the KV heads of a row into
// blocks, and which bytes of a token's scales each copy takes.
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

}  // namespace fp4
}  // namespace minisgl
